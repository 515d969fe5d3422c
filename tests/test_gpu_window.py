"""Windowed attention with sinks (GPU): forward and backward against the 64-bit formulas with derived bounds."""

import numpy as np
import pytest
import torch

import bf16_numerics_b200 as fa
from oracle import attention as A
from tests import plain64 as X

pytestmark = pytest.mark.gpu


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _heads(g, B, H, N, d, layout):
    if layout == "bhnd":
        return _normal(g, B, H, N, d)
    if layout == "bnhd":
        return _normal(g, B, N, H, d).transpose(1, 2)
    if layout == "fused":  # one of three slices of a projection: gaps between rows
        return _normal(g, B, N, 3, H, d)[:, :, 1].transpose(1, 2)
    assert layout == "hbnd"
    return _normal(g, H, B, N, d).transpose(0, 1)


def _inputs(B, H, Hkv, N, d, layout="bhnd", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_heads(g, B, H, N, d, layout), _heads(g, B, Hkv, N, d, layout), _heads(g, B, Hkv, N, d, layout),
            _heads(g, B, H, N, d, layout))


def _check(q, k, v, do, window, sinks, mode=fa.STABILIZED, beta=2.0):
    B, H, N, d = q.shape
    G = H // k.shape[1]
    o, lse, st = fa.window_attention_forward(q, k, v, window, sinks, mode, beta)
    dq, dk, dv, _ = fa.window_attention_backward(q, k, v, o, do, lse, st.m, window, sinks, mode, beta)
    torch.cuda.synchronize()
    status, word = fa.fa_device_error()
    assert status == 0, f"device error word {word:#x}"
    seen = X.visible(N, window, sinks, q.device)
    for b in range(B):
        for kv in range(k.shape[1]):
            sk = sv = bk = bv = 0
            for h in range(kv * G, (kv + 1) * G):
                f = X.attention(q[b, h], k[b, kv], v[b, kv], seen)
                X.assert_within("o", o[b, h], f["o"], X.rounded(f["o_bound"], f["o"]))
                X.assert_within("lse", lse[b, h], f["lse"], f["lse_bound"])
                r = X.gradients(q[b, h], k[b, kv], v[b, kv], o[b, h], do[b, h], f, f["lse_bound"])
                X.assert_within("dq", dq[b, h], r["dq"], X.rounded(r["dq_bound"], r["dq"]))
                sk, bk, sv, bv = sk + r["dk"], bk + r["dk_bound"], sv + r["dv"], bv + r["dv_bound"]
            X.assert_within("dk", dk[b, kv], sk, X.rounded(bk, sk))
            X.assert_within("dv", dv[b, kv], sv, X.rounded(bv, sv))
    return o, lse, st, dq, dk, dv


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [
    (1, 1, 0), (2, 1, 1), (127, 16, 0), (128, 128, 4), (129, 1, 0), (129, 2, 128), (200, 64, 3), (257, 300, 0),
    (384, 128, 129), (500, 129, 200), (640, 127, 1), (1000, 256, 0), (1025, 384, 130), (1300, 130, 1300),
    (1536, 2**31 - 1, 0), (900, 2**31 - 1, 2**31 - 1)])
def test_matches_the_formulas(cuda_device, d, N, window, sinks):
    _check(*_inputs(1, 2, 2, N, d, seed=N + window % 997 + d), window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (6, 2), (8, 8), (3, 3), (5, 1)])
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "fused", "hbnd"])
def test_shared_heads_and_strides(cuda_device, d, H, Hkv, layout):
    _check(*_inputs(2, H, Hkv, 333, d, layout, seed=H * 10 + Hkv), 100, 5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H,Hkv,window,sinks", [(5000, 4, 1, 700, 4), (4096, 2, 2, 4000, 0), (3333, 6, 2, 40, 260)])
def test_long_rows(cuda_device, d, N, H, Hkv, window, sinks):
    _check(*_inputs(1, H, Hkv, N, d, "bnhd", seed=7), window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", [fa.STANDARD, fa.STABILIZED, fa.STABILIZED_MARGIN])
def test_shift_rule_on_tied_rows(cuda_device, d, mode):
    """Keys repeated inside the window, in the sinks and across the two: rm, rs and m are the rule's, on scores that
    are exact in fp32 (a dyadic grid; d = 64) or near enough for the branch (d = 128)."""
    N, window, sinks = 520, 200, 6
    rng = np.random.default_rng(5)
    q, k, v, do = (torch.from_numpy(rng.integers(-4, 5, (1, 2, N, d)).astype(np.float32) / 4).to(torch.bfloat16).cuda()
                   for _ in range(4))
    k[:, :, 3] = k[:, :, 1]
    k[:, :, 300:400:7] = k[:, :, 2:3]
    o, lse, st, *_ = _check(q, k, v, do, window, sinks, mode)
    seen = X.visible(N, window, sinks, "cpu").numpy()
    for h in range(2):
        s = (q[0, h].double() @ k[0, h].double().T).cpu().numpy()
        s = np.where(seen, (s.astype(np.float32) * A.scale_f32(d)).astype(np.float32), -np.inf)
        rm = s.max(-1)
        rs = (s == rm[:, None]).sum(-1)
        assert np.array_equal(st.rs[0, h].cpu().numpy(), rs)
        assert np.array_equal(st.rm[0, h].cpu().numpy(), rm.astype(np.float32))
        assert np.array_equal(st.m[0, h].cpu().numpy(), A.select_shift(rm, rs, 2.0, mode))
    assert bool((st.rs > 1).any())
    if mode != fa.STANDARD:
        assert bool((st.pbar_max[st.rs > 1] < 1).all())


@pytest.mark.parametrize("d", [64, 128])
def test_wide_window_is_causal_attention(cuda_device, d):
    """With a window of the whole row the result is fa_fwd's: same statistics bit for bit, o and the gradients within
    a rounding (the tiles are visited in another order)."""
    q, k, v, do = _inputs(2, 3, 3, 777, d, seed=3)
    a = fa.window_attention_forward(q, k, v)
    b = fa.attention_forward(q, k, v)
    for name in ("rm", "rs", "m", "pbar_max"):
        assert torch.equal(getattr(a[2], name), getattr(b[2], name)), name
    assert (a[0].float() - b[0].float()).abs().max() <= 2 * 2.0 ** -8 * b[0].float().abs().max()
    ga = fa.window_attention_backward(q, k, v, b[0], do, b[1], b[2].m)
    gb = fa.attention_backward(q, k, v, b[0], do, b[1], b[2].m)
    for x, y in zip(ga[:3], gb[:3]):
        assert (x.float() - y.float()).abs().max() <= 2 * 2.0 ** -8 * y.float().abs().max()


def test_gradient_against_differences(cuda_device):
    """<dq, e> + <dk, e'> + <dv, e''> is the derivative of <o, do> along (e, e', e''), by central differences of the
    64-bit form; bf16 gradients carry 2^-8 of their size (measured as a norm) plus dS and P roundings of the same."""
    q, k, v, do = _inputs(1, 4, 2, 300, 64, seed=11)
    o, lse, st = fa.window_attention_forward(q, k, v, 50, 4)
    grads = fa.window_attention_backward(q, k, v, o, do, lse, st.m, 50, 4)[:3]
    g = torch.Generator(device="cuda").manual_seed(1)
    seen = X.visible(300, 50, 4, q.device)

    def value(t, dirs):
        qq, kk, vv = (x.double() + t * e for x, e in zip((q, k, v), dirs))
        kk, vv = kk.repeat_interleave(2, 1), vv.repeat_interleave(2, 1)
        return float((X.attention(qq, kk, vv, seen)["o"] * do.double()).sum())

    for _ in range(3):
        dirs = [torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64) for x in (q, k, v)]
        slope = (value(1e-4, dirs) - value(-1e-4, dirs)) / 2e-4
        got = sum(float((x.double() * e).sum()) for x, e in zip(grads, dirs))
        size = sum(float(x.double().norm()) for x in grads)  # a random direction projects with unit variance
        assert abs(got - slope) <= 4 * 3 * 2.0 ** -8 * size


@pytest.mark.parametrize("d", [64, 128])
def test_outputs_stay_inside_their_rows(cuda_device, d):
    """Outputs are slices of larger buffers: what lies between and behind the rows is left as it was."""
    B, H, Hkv, N = 2, 4, 2, 201
    q, k, v, do = _inputs(B, H, Hkv, N, d, seed=9)

    def slot(heads):
        whole = torch.full((B, N + 3, heads + 1, d + 8), 7.0, device="cuda", dtype=torch.bfloat16)
        return whole, whole[:, 1:N + 1, :heads, :d].transpose(1, 2)

    (wo, o), (wq, dq), (wk, dk), (wv, dv) = slot(H), slot(H), slot(Hkv), slot(Hkv)
    lse = torch.empty(B, H, N, device="cuda")
    st = fa.RowStats.empty(B, H, N, "cuda")
    size = fa.fa_window_bwd_workspace_bytes(B, H, Hkv, N, d, 64, 4)
    ws = torch.full((size + 512,), 0xA5, device="cuda", dtype=torch.uint8)
    fa.fa_window_fwd(q, k, v, o, lse, st, 64, 4)
    fa.fa_window_bwd(q, k, v, o, do, lse, st.m, dq, dk, dv, ws[256:256 + size], 64, 4)
    ref = fa.window_attention_forward(q, k, v, 64, 4)
    gref = fa.window_attention_backward(q, k, v, ref[0], do, ref[1], ref[2].m, 64, 4)
    assert torch.equal(o, ref[0]) and torch.equal(dk, gref[1]) and torch.equal(dv, gref[2])
    assert (dq.float() - gref[0].float()).abs().max() <= 2 * 2.0 ** -8 * gref[0].float().abs().max()
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + size:] == 0xA5).all())
    for whole, x in ((wo, o), (wq, dq), (wk, dk), (wv, dv)):
        x.fill_(7.0)
        assert bool((whole == 7.0).all())


@pytest.mark.parametrize("d", [64, 128])
def test_streams_and_graph(cuda_device, d):
    """Captured and replayed on new inputs beside an eager call on another stream, each with its own workspace."""
    first, second = _inputs(1, 4, 2, 400, d, seed=21), _inputs(1, 4, 2, 400, d, seed=22)

    def step(t, **kw):
        q, k, v, do = t
        o, lse, st = fa.window_attention_forward(q, k, v, 96, 8, **kw)
        dq, dk, dv, ws = fa.window_attention_backward(q, k, v, o, do, lse, st.m, 96, 8, **kw)
        return o, lse, dk, dv, dq

    ref1, ref2 = step(first), step(second)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    static = [t.clone() for t in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(static)
    for t, new in zip(static, second):
        t.copy_(new)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    graph.replay()
    eager = step(first, stream=other)
    torch.cuda.synchronize()
    for got, ref in ((out, ref2), (eager, ref1)):
        for a, b in zip(got[:4], ref[:4]):
            assert torch.equal(a, b)
        assert (got[4].float() - ref[4].float()).abs().max() <= 2 * 2.0 ** -8 * ref[4].float().abs().max()


def test_python_refuses_what_does_not_fit(cuda_device):
    q, k, v, do = _inputs(1, 4, 2, 70, 64)
    o, lse, st = fa.window_attention_forward(q, k, v, 8, 1)
    for args in ((q.float(), k, v), (q.cpu(), k, v), (q[0], k, v), (q, k[:, :, :9], v), (q, k, v[:, :1]), (q, k.float(), v),
                 (q, k, v.cpu()), (q.transpose(2, 3), k, v), (q, k[0], v)):
        with pytest.raises(ValueError):
            fa.window_attention_forward(*args, 8, 1)
        with pytest.raises(ValueError):
            fa.window_attention_backward(*args, o, do, lse, st.m, 8, 1)
    for i in range(3):
        args = [q, k, v]
        args[i] = "x"
        with pytest.raises(TypeError):
            fa.window_attention_forward(*args, 8, 1)
    for bad in (lse[:, :2], lse.half(), lse.cpu(), lse.transpose(1, 2)):
        with pytest.raises(ValueError):
            fa.fa_window_fwd(q, k, v, o, bad, None, 8, 1)
        with pytest.raises(ValueError):
            fa.window_attention_backward(q, k, v, o, do, bad, st.m, 8, 1)
        with pytest.raises(ValueError):
            fa.window_attention_backward(q, k, v, o, do, lse, bad, 8, 1)
        with pytest.raises(ValueError):
            fa.fa_window_fwd(q, k, v, o, lse, fa.RowStats(m=bad), 8, 1)
    with pytest.raises(ValueError):
        fa.fa_window_fwd(q, k, v, o, lse, fa.RowStats(rs=lse), 8, 1)
    for window, sinks in ((0, 0), (-1, 0), (2**31, 0), (2**32 + 5, 0), (4, -1), (4, 2**31)):
        with pytest.raises(ValueError):
            fa.window_attention_forward(q, k, v, window, sinks)
    for kw in (dict(softmax_mode=9), dict(beta=1.0), dict(beta=float("nan"))):
        with pytest.raises(fa.FaError):
            fa.window_attention_forward(q, k, v, 8, 1, **kw)
    with pytest.raises(fa.FaError) as e:
        fa.window_attention_backward(q, k, v, o, do, lse, None, 8, 1)  # a stabilised mode without its shift
    assert e.value.code == 1
    with pytest.raises(fa.FaError) as e:
        fa.window_attention_backward(q, k, v, o, do, lse, st.m, 8, 1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 3
    with pytest.raises(fa.FaError):  # a broadcast input: elements share memory
        fa.window_attention_forward(q, k[:, :1].expand(1, 2, 70, 64), v, 8, 1)
    o0, lse0, _ = fa.window_attention_forward(q[:, :, :0], k[:, :, :0], v[:, :, :0], 8, 1)
    assert o0.numel() == 0 and lse0.shape == (1, 4, 0)
    # partial statistics, and inputs that require gradients (the call records none)
    m = torch.empty(1, 4, 70, device="cuda")
    fa.fa_window_fwd(q, k, v, o, lse, fa.RowStats(m=m), 8, 1)
    assert torch.equal(m, st.m)
    o1, _, _ = fa.window_attention_forward(q.clone().requires_grad_(), k, v, 8, 1)
    assert torch.equal(o1, o) and not o1.requires_grad


def test_past_two_to_the_31_elements(cuda_device):
    """Tensors of more than 2^31 elements: the last rows of the last head, whose window reaches only their neighbours,
    against the formulas on a slice."""
    H, Hkv, N, d, window = 10, 5, 1_700_000, 128, 100
    assert H * N * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    make = lambda h: torch.randn(1, h, N, d, device="cuda", generator=g, dtype=torch.bfloat16)
    q, k, v, do = make(H), make(Hkv), make(Hkv), make(H)
    o, lse, st = fa.window_attention_forward(q, k, v, window)
    dq, dk, dv, ws = fa.window_attention_backward(q, k, v, o, do, lse, st.m, window)
    assert fa.fa_device_error() == (0, 0)
    n, m = 500, 300  # the last n rows hold the whole window of the last m
    for h in (0, H - 1):
        kv = h // 2
        seen = X.visible(n, window, 0, "cuda")
        sk = sv = bk = bv = 0
        for hh in (2 * kv, 2 * kv + 1):
            f = X.attention(q[0, hh, -n:], k[0, kv, -n:], v[0, kv, -n:], seen)
            r = X.gradients(q[0, hh, -n:], k[0, kv, -n:], v[0, kv, -n:], o[0, hh, -n:], do[0, hh, -n:], f, f["lse_bound"])
            sk, bk, sv, bv = sk + r["dk"], bk + r["dk_bound"], sv + r["dv"], bv + r["dv_bound"]
            if hh == h:
                X.assert_within("o", o[0, h, -m:], f["o"][-m:], X.rounded(f["o_bound"], f["o"])[-m:])
                X.assert_within("lse", lse[0, h, -m:], f["lse"][-m:], f["lse_bound"][-m:])
                X.assert_within("dq", dq[0, h, -m:], r["dq"][-m:], X.rounded(r["dq_bound"], r["dq"])[-m:])
        X.assert_within("dk", dk[0, kv, -m:], sk[-m:], X.rounded(bk, sk)[-m:])
        X.assert_within("dv", dv[0, kv, -m:], sv[-m:], X.rounded(bv, sv)[-m:])
