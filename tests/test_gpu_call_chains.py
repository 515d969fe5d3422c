"""Calls of different kinds after one another on one stream, with memory that goes from one to the next (GPU).

Launches overlap at their ends, so memory that an earlier call still uses must not be written before it has ended: a
scratch tensor that serves every call, and blocks that the allocator hands on when a call's own workspace or a caller's
temporaries are dropped.  Every output is compared with the same call on memory of its own, waited for.  All outputs
but dq are reproducible bit for bit; dq sums fp32 partials in an order that varies, so two of its values differ by less
than a bf16 step of the largest."""

import pytest
import torch

import bf16_numerics_b200 as fa
from tests import test_gpu_cached as C
from tests import test_gpu_window as W

pytestmark = pytest.mark.gpu

WINDOW, SINKS = 90, 5


class Chain:
    """A cached call with many parts to join, a windowed and a plain training step, and their results in isolation."""

    def __init__(self, d, T, G, ctx, N):
        Hkv, B = 2, len(ctx)
        self.H, self.Hkv, self.d, self.T, self.B, self.N = Hkv * G, Hkv, d, T, B, N
        self.cache = C.Cache(ctx, T, Hkv, d, 64, seed=d + T)
        g = torch.Generator(device="cuda").manual_seed(d)
        self.cq = C._normal(g, B, T, Hkv * G, d).transpose(1, 2)
        self.win = W._inputs(2, 4, 2, N, d, "bnhd", seed=1)
        self.full = W._inputs(1, 4, 4, N, d, seed=2)
        self.wf = fa.window_attention_forward(*self.win[:3], WINDOW, SINKS)
        self.pf = fa.attention_forward(*self.full[:3])
        torch.cuda.synchronize()
        self.ref = [self.attend(None)]
        torch.cuda.synchronize()
        self.ref.append(self.window(None))
        torch.cuda.synchronize()
        self.ref.append(self.plain(None))
        torch.cuda.synchronize()

    def scratch(self):
        size = max(fa.fa_cached_workspace_bytes(self.B, self.H, self.Hkv, self.T, self.d),
                   fa.fa_window_bwd_workspace_bytes(2, 4, 2, self.N, self.d, WINDOW, SINKS),
                   fa.fa_bwd_workspace_bytes(1, 4, self.N, self.d))
        return torch.empty(size, device="cuda", dtype=torch.uint8)

    def attend(self, ws):
        c = self.cache
        return fa.cached_attention(self.cq, c.k, c.v, c.table, c.ctx_len, workspace=ws)

    def window(self, ws):
        q, k, v, do = self.win
        o, lse, st = self.wf
        return fa.window_attention_backward(q, k, v, o, do, lse, st.m, WINDOW, SINKS, workspace=ws)[:3]

    def plain(self, ws):
        q, k, v, do = self.full
        o, lse, st = self.pf
        return fa.attention_backward(q, k, v, o, do, lse, st.m, workspace=ws)[:3]

    def check(self, which, out, note):
        ref = self.ref[which]
        if which == 0:
            assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), note
            return
        assert torch.equal(out[1], ref[1]) and torch.equal(out[2], ref[2]), note
        diff, top = (out[0].float() - ref[0].float()).abs().max(), ref[0].float().abs().max()
        assert diff <= 2 * 2.0 ** -8 * top, (note, float(diff), float(top))


CHAINS = [(64, 1, 4, [30000, 12000, 500], 300), (128, 1, 4, [30000, 12000, 500], 300),
          (64, 40, 8, [9000, 6000], 700), (128, 40, 8, [9000, 6000], 700)]
ORDERS = [(0, 1, 0, 2, 0), (0, 0, 2, 1, 0, 1)]


@pytest.mark.parametrize("d,T,G,ctx,N", CHAINS)
@pytest.mark.parametrize("order", ORDERS)
def test_one_scratch_tensor_for_every_call(cuda_device, d, T, G, ctx, N, order):
    chain = Chain(d, T, G, ctx, N)
    ws = chain.scratch()
    call = (chain.attend, chain.window, chain.plain)
    for rep in range(12):
        out = [call[which](ws) for which in order]
        torch.cuda.synchronize()
        for at, (which, x) in enumerate(zip(order, out)):
            chain.check(which, x, (rep, at, which))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [call[which](ws) for which in order]
    for rep in range(6):
        graph.replay()
        torch.cuda.synchronize()
        for at, (which, x) in enumerate(zip(order, out)):
            chain.check(which, x, ("graph", rep, at, which))
    assert fa.fa_device_error() == (0, 0)


@pytest.mark.parametrize("d,T,G,ctx,N", CHAINS)
def test_blocks_handed_on_by_the_allocator(cuda_device, d, T, G, ctx, N):
    """Workspaces of the calls' own, and a forward's temporaries, dropped before the next call allocates."""
    chain = Chain(d, T, G, ctx, N)
    wf, pf = [t.clone() for t in chain.wf[:2]], [t.clone() for t in chain.pf[:2]]
    new = C._normal(torch.Generator(device="cuda").manual_seed(3), chain.B, chain.Hkv, T, d)
    pool = [chain.cache.k.clone(), chain.cache.v.clone()]
    written = [p.clone() for p in pool]
    fa.fa_cache_append(new, new, *written, chain.cache.table, chain.cache.ctx_len)
    torch.cuda.synchronize()
    for rep in range(12):
        out = [(0, chain.attend(None)), (1, chain.window(None)), (0, chain.attend(None)), (2, chain.plain(None))]
        tmp = [t.clone() for t in chain.win[:3]]
        a = fa.window_attention_forward(*tmp, WINDOW, SINKS, with_stats=False)[:2]
        del tmp
        out.append((1, chain.window(None)))
        tmp = [t.clone() for t in chain.full[:3]]
        b = fa.attention_forward(*tmp, with_stats=False)[:2]
        del tmp
        out.append((2, chain.plain(None)))
        tmp = [new.clone(), new.clone()]
        fa.fa_cache_append(*tmp, *pool, chain.cache.table, chain.cache.ctx_len)
        del tmp
        out.append((1, chain.window(None)))
        torch.cuda.synchronize()
        for at, (which, x) in enumerate(out):
            chain.check(which, x, (rep, at, which))
        for got, ref in ((a, wf), (b, pf)):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), rep
        for got, ref, old in zip(pool, written, (chain.cache.k, chain.cache.v)):
            assert torch.equal(torch.nan_to_num(got, 9.0), torch.nan_to_num(ref, 9.0)), rep
            got.copy_(old)
    assert fa.fa_device_error() == (0, 0)
