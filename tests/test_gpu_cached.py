"""Attention over a paged cache, and the cache's writes (GPU), against the 64-bit formulas with derived bounds.

Every pool starts as NaN, so a slot that should not count but does shows up; table entries that a call has no need of
hold page ids outside the pool."""

import math

import numpy as np
import pytest
import torch

import bf16_numerics_b200 as fa
from bf16_numerics_b200 import _abi
from tests import plain64 as X

pytestmark = pytest.mark.gpu

INF = fa.NO_WINDOW


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _words(kind, B, T, rng):
    """bool [B, T, T]: which new tokens each sees."""
    sees = np.zeros((B, T, T), bool)
    for b in range(B):
        for u in range(T):
            if kind == "chain":
                sees[b, u, :u + 1] = True
            elif kind == "star":
                sees[b, u, [0, u]] = True
            else:
                if u:
                    sees[b, u] = sees[b, rng.integers(0, u)]
                sees[b, u, u] = True
        if kind == "absent":
            sees[b, rng.random(T) < 0.4] = False
            if b == 0:
                sees[b] = False
    return sees


def _pack(sees):
    T = sees.shape[-1]
    return torch.from_numpy((sees.astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(-1, dtype=np.uint64)
                            .view(np.int64)).cuda()


def _visible(sees, ctx, window, sinks):
    """bool [T, ctx + T] for one sequence."""
    T = sees.shape[0]
    stands = np.concatenate([np.arange(ctx), ctx + sees.sum(-1) - 1])
    seen = np.concatenate([np.ones((T, ctx), bool), sees], -1)
    for t in range(T):
        seen[t] &= (stands[ctx + t] - stands < window) | (stands < sinks)
    return seen & sees.any(-1)[:, None]


class Cache:
    def __init__(self, ctx, T, Hkv, d, page, seed=0, window=INF, sinks=0, sees=None, spare=2, num_pages=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, B = list(ctx), len(ctx)
        width = max(1, -(-(max(ctx) + T) // page)) + 1
        used = sum(-(-(c + T) // page) for c in ctx)
        P = num_pages or used + spare
        make = torch.full if num_pages is None else (lambda s, v, **k: torch.empty(s, **k))
        self.k, self.v = (make((P, Hkv, page, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        ids = P - 1 - rng.permutation(used) if num_pages else rng.permutation(P)[:used]
        table = np.full((B, width), P + 5)
        at = 0
        self.rows = []
        for b, c in enumerate(ctx):
            n = -(-(c + T) // page)
            table[b, :n] = ids[at:at + n]
            at += n
            k, v = _normal(g, Hkv, c + T, d), _normal(g, Hkv, c + T, d)
            self.rows.append((k, v))
            live = np.arange(c + T)
            if sees is not None:
                live = live[np.concatenate([np.ones(c, bool), sees[b].any(0)])]
            to = torch.from_numpy(table[b][live // page].astype(np.int64)).cuda()
            off, live = torch.from_numpy(live % page).cuda(), torch.from_numpy(live).cuda()
            self.k[to, :, off] = k[:, live].transpose(0, 1)
            self.v[to, :, off] = v[:, live].transpose(0, 1)
            for i in range(n):  # pages that no token sees any more
                if (i + 1) * page <= c - window + 1 and i * page >= sinks:
                    table[b, i] = -1 - i
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.ctx_len = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")


def _check(cache, q, sees, window, sinks, o, lse):
    B, H, T, d = q.shape
    Hkv = cache.k.shape[1]
    G = H // Hkv
    for b, c in enumerate(cache.ctx):
        seen = torch.from_numpy(_visible(sees[b], c, window, sinks)).cuda()
        k, v = cache.rows[b]
        f = X.attention(q[b], k.repeat_interleave(G, 0), v.repeat_interleave(G, 0), seen)
        X.assert_within(f"o of {b}", o[b], f["o"], X.rounded(f["o_bound"], f["o"]))
        X.assert_within(f"lse of {b}", lse[b], f["lse"], f["lse_bound"])


def _run(ctx, T, H, Hkv, d, page, window=INF, sinks=0, kind="chain", mode=fa.STABILIZED, seed=0, **kw):
    rng = np.random.default_rng(seed)
    sees = _words(kind, len(ctx), T, rng)
    cache = Cache(ctx, T, Hkv, d, page, seed, window, sinks, sees, **kw)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = _normal(g, len(ctx), T, H, d).transpose(1, 2)
    o, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len,
                                 None if kind == "chain" else _pack(sees), window, sinks, mode)
    status, word = fa.fa_device_error()
    assert status == 0, f"device error word {word:#x}"
    _check(cache, q, sees, window, sinks, o, lse)
    return cache, q, o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T,H,Hkv", [(1, 1, 1), (1, 8, 2), (3, 6, 6), (13, 4, 2), (64, 3, 1)])
def test_lengths_and_pages(cuda_device, d, page, T, H, Hkv):
    _run([0, 1, 15, 127, 128, 129, 300, 1000], T, H, Hkv, d, page, seed=page + T)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 7), (8, 4), (9, 4), (16, 4), (17, 4), (33, 3), (64, 2), (64, 8), (43, 5), (1, 128),
                                 (2, 100)])
def test_rows_of_a_key_head(cuda_device, d, T, G):
    """Four, two and one copies of the rows, several row tiles, the last of them ragged."""
    _run([700, 5, 333], T, 2 * G, 2, d, 64, kind="tree", seed=T * G)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (5, 0), (64, 3), (100, 130), (128, 16), (129, 0), (300, 500),
                                          (INF, INF), (4, 100000)])
@pytest.mark.parametrize("kind", ["chain", "tree", "star", "absent"])
def test_windows_and_trees(cuda_device, d, window, sinks, kind):
    _run([0, 3, 200, 640, 1111], 11, 4, 2, d, 32, window, sinks, kind, seed=window % 1000 + sinks % 1000)


@pytest.mark.parametrize("T", [2, 3, 7])
def test_window_as_long_as_the_tree(cuda_device, T):
    """A token may name an absent one, which stands one place before the root: T places away at most."""
    for window in (T - 1, T, T + 1):
        for seed in range(4):
            _run([176, 28, 90, 5, 0], T, 4, 2, 64, 32, window, seed % 3, "absent", seed=seed)


@pytest.mark.parametrize("d", [64, 128])
def test_long_context_is_split_and_joined(cuda_device, d):
    _run([40000], 1, 2, 1, d, 128, seed=1)
    _run([30011, 12, 0, 9000], 7, 4, 2, d, 64, kind="tree", seed=2)
    _run([20000], 4, 2, 1, d, 16, window=9000, sinks=200, kind="tree", seed=3)


def test_many_sequences(cuda_device):
    rng = np.random.default_rng(4)
    _run([int(x) for x in rng.integers(0, 600, 150)], 2, 4, 2, 64, 16, seed=4)


@pytest.mark.parametrize("mode", [fa.STANDARD, fa.STABILIZED, fa.STABILIZED_MARGIN])
def test_tied_rows(cuda_device, mode):
    """Repeated keys (tied maxima, positive and negative) under each shift rule."""
    cache = Cache([500, 77], 2, 2, 64, 32, seed=6)
    for b, c in enumerate(cache.ctx):
        k, v = cache.rows[b]
        k[:, 5::9] = k[:, 5:6]
        for j in range(5, c + 2, 9):
            cache.k[int(cache.table[b, j // 32]), :, j % 32] = k[:, 5]
    g = torch.Generator(device="cuda").manual_seed(7)
    base = cache.rows[0][0][:, 5]  # rows along the repeated key, and against it
    q = torch.stack([base, -base], 1).unsqueeze(0).repeat(2, 1, 1, 1) * 2 + _normal(g, 2, 2, 2, 64) / 8
    o, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len, softmax_mode=mode)
    _check(cache, q, _words("chain", 2, 2, None), INF, 0, o, lse)


def test_pages_past_two_to_the_31(cuda_device):
    """Pages whose offsets in the pool do not fit in 32 bits."""
    pages = 2 ** 31 // (2 * 256 * 128) + 64
    cache, q, o, lse = _run([900, 40], 4, 4, 2, 128, 256, kind="tree", num_pages=pages)
    k, v = _normal(torch.Generator(device="cuda").manual_seed(1), 2, 2, 4, 128), q[:, :2]
    fa.fa_cache_append(k, v, cache.k, cache.v, cache.table, cache.ctx_len)
    for b, c in enumerate(cache.ctx):
        for t in range(4):
            page = int(cache.table[b, (c + t) // 256])
            assert page * 2 * 256 * 128 > 2 ** 31 - 2 ** 24
            assert torch.equal(cache.k[page, :, (c + t) % 256], k[b, :, t])
            assert torch.equal(cache.v[page, :, (c + t) % 256], v[b, :, t])


def test_lengths_and_ids_outside_the_cache_are_reported(cuda_device):
    cache = Cache([100, 60, 300], 2, 2, 64, 16, seed=8)
    q = _normal(torch.Generator(device="cuda").manual_seed(9), 3, 4, 2, 64)
    sees = _words("chain", 3, 2, None)
    good = cache.ctx_len.clone()
    for bad in (-1, 10 ** 9, 2 ** 31 - 1, cache.table.shape[1] * 16 - 1):
        cache.ctx_len[1] = bad
        o, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len)
        status, word = fa.fa_device_error()
        assert status == _abi.FA_ERR_BAD_PAGE and word == (6 << 24 | 1 << 16 | 1)
        assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())
        keep = Cache.__new__(Cache)
        keep.ctx, keep.rows, keep.k = [100, 300], [cache.rows[0], cache.rows[2]], cache.k
        _check(keep, q[[0, 2]], sees, INF, 0, o[[0, 2]], lse[[0, 2]])
    cache.ctx_len.copy_(good)
    for bad in (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = cache.table.clone()
        table[2, 3] = bad
        o, lse = fa.cached_attention(q, cache.k, cache.v, table, cache.ctx_len)
        status, word = fa.fa_device_error()
        assert status == _abi.FA_ERR_BAD_PAGE and word == (6 << 24 | 2 << 16 | 2)
        assert bool(torch.isfinite(lse).all())
        before = [cache.k.clone(), cache.v.clone()]
        at = torch.tensor([10, 10, 48], dtype=torch.int32, device="cuda")  # only sequence 2's write meets the bad entry
        new = _normal(torch.Generator(device="cuda").manual_seed(1), 3, 2, 1, 64)
        fa.fa_cache_append(new, new, cache.k, cache.v, table, at)
        assert fa.fa_device_error()[1] == (6 << 24 | 4 << 16 | 2)
        for pool, old in zip((cache.k, cache.v), before):
            for b in (0, 1):
                old[int(table[b, 0]), :, 10] = new[b, :, 0]
            assert torch.equal(torch.nan_to_num(pool), torch.nan_to_num(old))
    assert fa.fa_device_error() == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hkv,page", [(1, 1, 16), (1, 12, 16), (5, 3, 32), (300, 2, 64), (1000, 1, 256)])
def test_append(cuda_device, d, T, Hkv, page):
    ctx = [0, 7, 200, 131]
    g = torch.Generator(device="cuda").manual_seed(T)
    for count in (None, [0, T, max(1, T // 2), 1]):
        cache = Cache(ctx, T, Hkv, d, page, seed=3)
        k, v = _normal(g, 4, T, Hkv, d).transpose(1, 2), _normal(g, 4, Hkv, T, d)
        want = [cache.k.clone(), cache.v.clone()]
        for b, c in enumerate(ctx):
            for t in range(T if count is None else count[b]):
                at = int(cache.table[b, (c + t) // page]), (c + t) % page
                want[0][at[0], :, at[1]] = k[b, :, t]
                want[1][at[0], :, at[1]] = v[b, :, t]
        n = None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda")
        fa.fa_cache_append(k, v, cache.k, cache.v, cache.table, cache.ctx_len, n)
        assert fa.fa_device_error() == (0, 0)
        for got, ref in zip((cache.k, cache.v), want):
            assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(ref, 9.0))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("M,Hkv,page", [(1, 1, 16), (5, 3, 16), (64, 2, 32), (33, 16, 256)])
def test_compact(cuda_device, d, M, Hkv, page):
    """Paths in order, other orders and repeated rows; nothing else moves."""
    rng = np.random.default_rng(M)
    ctx = [0, 9, 250, 100]
    cache = Cache(ctx, 64, Hkv, d, page, seed=2)
    src = np.stack([np.sort(rng.permutation(64)[:M]), rng.permutation(64)[:M], rng.integers(0, 64, M), np.arange(M)])
    count = [M, M, max(1, M - 1), M]
    want = [cache.k.clone(), cache.v.clone()]
    for b, c in enumerate(ctx):
        for i in range(count[b]):
            j = c + int(src[b, i])
            for pool, old in zip(want, (cache.k, cache.v)):
                pool[int(cache.table[b, (c + i) // page]), :, (c + i) % page] = \
                    old[int(cache.table[b, j // page]), :, j % page]
    fa.fa_cache_compact(cache.k, cache.v, cache.table, cache.ctx_len,
                        torch.from_numpy(src.astype(np.int32)).cuda(), torch.tensor(count, dtype=torch.int32).cuda())
    assert fa.fa_device_error() == (0, 0)
    for got, ref in zip((cache.k, cache.v), want):
        assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(ref, 9.0))


def test_compact_and_append_report_bad_counts(cuda_device):
    cache = Cache([20, 30], 8, 2, 64, 16, seed=2)
    before = cache.k.clone()
    src = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    for count, word in (([-1, 0], 6 << 24 | 5 << 16), ([0, 5], 6 << 24 | 5 << 16 | 1)):
        fa.fa_cache_compact(cache.k, cache.v, cache.table, cache.ctx_len, src, torch.tensor(count, dtype=torch.int32).cuda())
        assert fa.fa_device_error() == (_abi.FA_ERR_BAD_PAGE, word)
    src[1, 1] = -3
    fa.fa_cache_compact(cache.k, cache.v, cache.table, cache.ctx_len, src, torch.tensor([0, 2], dtype=torch.int32).cuda())
    assert fa.fa_device_error() == (_abi.FA_ERR_BAD_PAGE, 6 << 24 | 6 << 16 | 1)
    new = _normal(torch.Generator(device="cuda").manual_seed(1), 2, 2, 3, 64)
    fa.fa_cache_append(new, new, cache.k, cache.v, cache.table, cache.ctx_len, torch.tensor([4, 0], dtype=torch.int32).cuda())
    assert fa.fa_device_error() == (_abi.FA_ERR_BAD_PAGE, 6 << 24 | 3 << 16)
    assert torch.equal(torch.nan_to_num(cache.k, 9.0), torch.nan_to_num(before, 9.0))


def test_outputs_stay_inside_their_rows(cuda_device):
    cache = Cache([130, 0, 70], 5, 2, 128, 32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(2)
    q = _normal(g, 3, 6, 5, 128)
    whole = torch.full((3, 7, 8, 136), 7.0, device="cuda", dtype=torch.bfloat16)
    o = whole[:, 1:6, 1:7, :128].transpose(1, 2)
    guard = torch.full((3 * 6 * 5 + 8,), 7.0, device="cuda")
    lse = guard[4:-4].view(3, 6, 5)
    size = fa.fa_cached_workspace_bytes(3, 6, 2, 5, 128)
    ws = torch.full((size + 512,), 0xA5, device="cuda", dtype=torch.uint8)
    fa.fa_cached_fwd(q, cache.k, cache.v, cache.table, cache.ctx_len, None, o, lse, ws[256:256 + size])
    _check(cache, q, _words("chain", 3, 5, None), INF, 0, o, lse)
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + size:] == 0xA5).all())
    o.fill_(7.0)
    assert bool((whole == 7.0).all()) and bool((guard[:4] == 7.0).all()) and bool((guard[-4:] == 7.0).all())


def test_replayed_graph_follows_the_lengths(cuda_device):
    """One capture of append + attention + compaction, replayed while the context grows, beside eager calls on another
    stream; every step against the formulas."""
    H, Hkv, T, d, page = 4, 2, 6, 64, 16
    cache = Cache([100, 17], 60, Hkv, d, page, seed=12)
    other = Cache([333, 4], T, Hkv, d, page, seed=13)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = _normal(g, 2, H, T, d), _normal(g, 2, Hkv, T, d), _normal(g, 2, Hkv, T, d)
    words = torch.zeros(2, T, dtype=torch.int64, device="cuda")
    src = torch.zeros(2, T, dtype=torch.int32, device="cuda")
    taken = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step():
        fa.fa_cache_append(k, v, cache.k, cache.v, cache.table, cache.ctx_len)
        out = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len, words, 50, 3)
        fa.fa_cache_compact(cache.k, cache.v, cache.table, cache.ctx_len, src, taken)
        cache.ctx_len.add_(taken)
        return out

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    side = torch.cuda.Stream()
    rng = np.random.default_rng(5)
    for _ in range(6):
        sees = _words("tree", 2, T, rng)
        words.copy_(_pack(sees))
        for t in (q, k, v):
            t.copy_(_normal(g, *t.shape))
        path = sees[:, T - 1]
        src.copy_(torch.from_numpy(np.argsort(~path, -1, kind="stable").astype(np.int32)))
        taken.copy_(torch.from_numpy(path.sum(-1).astype(np.int32)))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        oo, ll = fa.cached_attention(q, other.k, other.v, other.table, other.ctx_len, stream=side)
        torch.cuda.synchronize()
        now = Cache.__new__(Cache)
        now.k, now.ctx = cache.k, cache.ctx
        now.rows = [tuple(torch.cat([x[:, :c], y[b]], 1) for x, y in zip(cache.rows[b], (k, v)))
                    for b, c in enumerate(cache.ctx)]
        _check(now, q, sees, 50, 3, o, lse)
        _check(other, q, _words("chain", 2, T, None), INF, 0, oo, ll)
        for b, c in enumerate(cache.ctx):  # the accepted path is now context
            at = torch.from_numpy(np.flatnonzero(path[b])).cuda()
            cache.rows[b] = tuple(torch.cat([x[:, :c], y[b][:, at]], 1) for x, y in zip(cache.rows[b], (k, v)))
            cache.ctx[b] = c + len(at)
    assert fa.fa_device_error() == (0, 0)


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_then_tokens(cuda_device, d):
    """The operators as a model would use them: a windowed prompt, its keys and values written to pages, then token by
    token over the cache -- the same rows as one windowed call over the whole text."""
    B, H, Hkv, N, n0, window, sinks, page = 2, 6, 2, 230, 200, 90, 5, 16
    g = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = _normal(g, B, N, H, d).transpose(1, 2), _normal(g, B, Hkv, N, d), _normal(g, B, Hkv, N, d)
    o, lse, _ = fa.window_attention_forward(q, k, v, window, sinks)
    first = fa.window_attention_forward(q[:, :, :n0], k[:, :, :n0], v[:, :, :n0], window, sinks)
    assert torch.equal(first[0], o[:, :, :n0]) and torch.equal(first[1], lse[:, :, :n0])
    width = -(-N // page)
    table = torch.randperm(B * width, device="cuda", generator=g).view(B, width).int()
    kp, vp = (torch.full((B * width, Hkv, page, d), math.nan, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.fa_cache_append(k[:, :, :n0], v[:, :, :n0], kp, vp, table, at)
    at += n0
    n = n0
    while n < N:
        T = min(1 + n % 4, N - n)
        fa.fa_cache_append(k[:, :, n:n + T], v[:, :, n:n + T], kp, vp, table, at)
        co, cl = fa.cached_attention(q[:, :, n:n + T], kp, vp, table, at, None, window, sinks)
        for b in range(B):
            seen = X.visible(N, window, sinks, q.device)[n:n + T]
            f = X.attention(q[b, :, n:n + T], k[b].repeat_interleave(H // Hkv, 0), v[b].repeat_interleave(H // Hkv, 0), seen)
            for x, y in ((co, cl), (o[:, :, n:n + T], lse[:, :, n:n + T])):
                X.assert_within("o", x[b], f["o"], X.rounded(f["o_bound"], f["o"]))
                X.assert_within("lse", y[b], f["lse"], f["lse_bound"])
        at += T
        n += T


def test_python_refuses_what_does_not_fit(cuda_device):
    cache = Cache([20, 30], 4, 2, 64, 16, seed=2)
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k = _normal(g, 2, 4, 3, 64), _normal(g, 2, 2, 3, 64)
    words = torch.ones(2, 3, dtype=torch.int64, device="cuda")
    src, count = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(fa.fa_cached_workspace_bytes(2, 4, 2, 3, 64), dtype=torch.uint8, device="cuda")
    good = dict(q=q, k_pages=cache.k, v_pages=cache.v, page_table=cache.table, ctx_len=cache.ctx_len, tree=words,
                workspace=ws)
    fa.cached_attention(**good)
    wide = torch.zeros(2, 4, 3, 128, dtype=torch.bfloat16, device="cuda")
    for name, bad in (("q", q.float()), ("q", q.cpu()), ("q", q[0]), ("q", wide[..., ::2]), ("q", q[:1]),
                      ("k_pages", cache.k.float()), ("k_pages", cache.k[0]), ("v_pages", cache.v[:1]),
                      ("v_pages", cache.v.cpu()), ("v_pages", cache.v.transpose(2, 3)), ("page_table", cache.table.long()),
                      ("page_table", cache.table[0]), ("page_table", cache.table.t()), ("ctx_len", cache.ctx_len[:1]),
                      ("ctx_len", cache.ctx_len.cpu()), ("tree", words[:, :2]), ("tree", words.int()),
                      ("workspace", ws.float()), ("workspace", ws.view(1, -1))):
        with pytest.raises(ValueError):
            fa.cached_attention(**{**good, name: bad})
    for name in ("q", "k_pages", "v_pages", "page_table", "ctx_len", "tree", "workspace"):
        with pytest.raises(TypeError):
            fa.cached_attention(**{**good, name: 3})
    for kw in (dict(window=0), dict(window=2**31), dict(sinks=-1), dict(sinks=2**40)):
        with pytest.raises(ValueError):
            fa.cached_attention(**good, **kw)
    for kw in (dict(window=1.5), dict(window=None), dict(beta="2")):
        with pytest.raises(TypeError):
            fa.cached_attention(**good, **kw)
    for kw in (dict(softmax_mode=7), dict(softmax_mode=2**40), dict(beta=1.0), dict(beta=math.inf)):
        with pytest.raises(fa.FaError) as e:
            fa.cached_attention(**good, **kw)
        assert e.value.code == _abi.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FaError) as e:
        fa.cached_attention(**{**good, "workspace": ws[:-1]})
    assert e.value.code == _abi.FA_ERR_WORKSPACE
    with pytest.raises(fa.FaError) as e:  # more than 64 new tokens
        fa.cached_attention(_normal(g, 2, 4, 65, 64), cache.k, cache.v, cache.table, cache.ctx_len)
    assert e.value.code == _abi.FA_ERR_UNSUPPORTED
    for args in ((k, k[:, :, :2], None), (k.float(), k, None), (k, k, count.long()), (k, k, count[:1]), (q, q, None)):
        with pytest.raises(ValueError):
            fa.fa_cache_append(args[0], args[1], cache.k, cache.v, cache.table, cache.ctx_len, args[2])
    for args in ((src.long(), count), (src[:1], count), (src, count[:1]), (src[0], count)):
        with pytest.raises(ValueError):
            fa.fa_cache_compact(cache.k, cache.v, cache.table, cache.ctx_len, *args)
    with pytest.raises(ValueError):
        fa.fa_cached_fwd(q, cache.k, cache.v, cache.table, cache.ctx_len, None, q[:, :2], torch.empty(2, 4, 3, device="cuda"), ws)
    with pytest.raises(ValueError):
        fa.fa_cached_fwd(q, cache.k, cache.v, cache.table, cache.ctx_len, None, q, torch.empty(2, 4, 3), ws)
    # nothing to do, and a full pool of arguments all the same
    o, lse = fa.cached_attention(q[:, :, :0], cache.k, cache.v, cache.table, cache.ctx_len)
    assert o.shape == (2, 4, 0, 64) and lse.shape == (2, 4, 0)
    assert fa.fa_device_error() == (0, 0)


@pytest.mark.parametrize("T,H,Hkv,d", [(1, 2, 1, 64), (9, 4, 1, 128), (64, 2, 1, 128), (48, 8, 1, 64)])
def test_withheld_arrive_ends_in_timeout(cuda_device, T, H, Hkv, d):
    """The bounded-wait exit of the split kernel in each of its forms (four, two and one copies of the rows, pairs of row
    tiles): a hook withholds an arrive that nothing else gives, the call ends with FA_ERR_TIMEOUT, and the next
    normal call on the same context is right."""
    cache = Cache([900], T, Hkv, d, 64, seed=1)
    q = _normal(torch.Generator(device="cuda").manual_seed(2), 1, H, T, d)
    torch.cuda.synchronize()
    assert fa.fa_device_error() == (0, 0)
    try:
        fa.fa_debug_set_wait_limit_ns(50_000_000)  # 50 ms: far above every legitimate wait here
        fa.fa_debug_inject_stall(_abi.FA_ERRWORD_CACHED)
        fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len)
        status, word = fa.fa_device_error()
    finally:
        fa.fa_debug_inject_stall(0)
        fa.fa_debug_set_wait_limit_ns(0)
    assert status == _abi.FA_ERR_TIMEOUT and word >> 24 == _abi.FA_ERRWORD_CACHED and word & 0xFFFF == 0
    o, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len)
    assert fa.fa_device_error() == (0, 0)
    _check(cache, q, _words("chain", 1, T, None), INF, 0, o, lse)
