"""Pages that a cached call has no need of (GPU): their table entries may hold anything -- ids outside the pool, or pages full
of NaN -- and nothing is reported; the entry of a page that some row sees is."""

import numpy as np
import pytest
import torch

import bf16_numerics_b200 as fa
from bf16_numerics_b200 import _abi
from tests import test_gpu_cached as C

pytestmark = pytest.mark.gpu


def _sees(kind, B, T):
    """bool [B, T, T]: trees with absent tokens (rows of False)."""
    sees = np.zeros((B, T, T), bool)
    for b in range(B):
        here = np.ones(T, bool)
        if kind == "behind":
            here[max(1, T // 4):] = False
        elif kind == "between":
            here[T // 4:3 * T // 4] = False
        elif kind == "nobody":
            here[:] = b > 0
        else:  # the root is absent, though all others name it: nobody stands at its place
            assert kind == "rootless"
            here[0] = False
        for u in np.flatnonzero(here):
            sees[b, u, :u + 1] = here[:u + 1]
            if kind == "rootless":
                sees[b, u, 0] = True
    return sees


def _needless(sees, ctx, page, window, sinks, width):
    """bool [width]: pages without a slot that a row sees or of a token that a word names."""
    T = sees.shape[0]
    need = np.zeros(width * page, bool)
    need[:ctx + T] = C._visible(sees, ctx, window, sinks).any(0)
    need[ctx:ctx + T] |= sees.any(0)
    return ~need.reshape(width, page).any(1)


def _call(kind, ctx, T, H, Hkv, d, page, window, sinks, fill, seed=0):
    sees = _sees(kind, len(ctx), T)
    cache = C.Cache(ctx, T, Hkv, d, page, seed, C.INF, 0, sees)
    q = C._normal(torch.Generator(device="cuda").manual_seed(seed + 1), len(ctx), T, H, d).transpose(1, 2)
    table = cache.table.cpu().numpy()
    spare = int(np.setdiff1d(np.arange(cache.k.shape[0]), table)[0])
    assert bool(torch.isnan(cache.k[spare]).all())
    put = {"outside": [-1, 2**31 - 1, cache.k.shape[0], -2**31], "nan": [spare]}[fill]
    count = 0
    for b, c in enumerate(ctx):
        for i in np.flatnonzero(_needless(sees[b], c, page, window, sinks, table.shape[1])):
            table[b, i] = put[count % len(put)]
            count += 1
    cache.table.copy_(torch.from_numpy(table))
    o, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len, C._pack(sees), window, sinks)
    assert fa.fa_device_error() == (0, 0)
    C._check(cache, q, sees, window, sinks, o, lse)
    return cache, q, sees


@pytest.mark.parametrize("fill", ["outside", "nan"])
@pytest.mark.parametrize("kind", ["behind", "between", "nobody", "rootless"])
@pytest.mark.parametrize("T,H,Hkv,d", [(17, 2, 2, 64), (20, 4, 2, 128), (60, 2, 2, 128), (64, 4, 2, 64), (64, 6, 2, 128)])
def test_pages_that_no_row_sees(cuda_device, T, H, Hkv, d, kind, fill):
    """Four, two and one copies of the rows, one and two row tiles."""
    for page in (16, 64):
        for window, sinks in ((C.INF, 0), (70, 0), (33, 20), (1, 0)):
            _call(kind, [0, 5, 130, 250, 767], T, H, Hkv, d, page, window, sinks, fill, seed=page + window % 99)


@pytest.mark.parametrize("fill", ["outside", "nan"])
def test_nobody_stands_at_the_root(cuda_device, fill):
    """The window of every row begins behind a page that a row at the root's place would see the last slot of."""
    for ctx, window in ((160, 17), (160, 33), (200, 9), (200, 57)):
        assert (ctx + 1 - window) % 16 == 0
        for first in (ctx - 1, ctx):  # the page boundary itself, and one slot before it
            _call("rootless", [first, 40], 5, 4, 2, 64, 16, window, 0, fill)


def test_the_page_of_a_named_token_is_needed(cuda_device):
    """Token 20 is absent, but token 3 names it: its page is looked up, and its bad id reported."""
    cache, q, sees = _call("behind", [100], 40, 2, 2, 64, 16, C.INF, 0, "outside")
    at = (100 + 20) // 16
    assert int(cache.table[0, at]) not in range(cache.k.shape[0])
    sees[0, 3, 20] = True
    _, lse = fa.cached_attention(q, cache.k, cache.v, cache.table, cache.ctx_len, C._pack(sees))
    assert fa.fa_device_error() == (_abi.FA_ERR_BAD_PAGE, _abi.FA_ERRWORD_CACHE_PAGE << 24 | 2 << 16)
    assert bool(torch.isfinite(lse[:, :, :10]).all())
