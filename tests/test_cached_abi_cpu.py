"""What the calls on a paged cache refuse (no GPU: refused before anything is launched)."""

import ctypes

import pytest
import torch

import bf16_numerics_b200 as fa
from bf16_numerics_b200 import _abi
from bf16_numerics_b200.build import build_library

BAD, UNSUPPORTED, WORKSPACE = _abi.FA_ERR_INVALID_ARG, _abi.FA_ERR_UNSUPPORTED, _abi.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def view(B, H, N, d, ptr=0x100000, strides=None):
    return ctypes.byref(_abi.FaView(ptr, *(strides or (H * N * d, N * d, d))))


def attend(lib, kp=0x1000, vp=0x1000, table=0x1000, ctx=0x1000, tree=None, lse=0x1000, ws=0x1000, ws_bytes=1 << 40,
           B=2, H=4, Hkv=2, T=3, d=64, pages=10, page=16, width=8, window=100, sinks=0, mode=1, beta=2.0, q=None, o=None):
    return lib.fa_cached_fwd(q or view(B, H, T, d), kp, vp, table, ctx, tree, o or view(B, H, T, d), lse, ws, ws_bytes,
                             B, H, Hkv, T, d, pages, page, width, window, sinks, mode, beta, None)


def test_attention_arguments(lib):
    for kw in (dict(window=0), dict(sinks=-1), dict(mode=5), dict(beta=1.0), dict(Hkv=3), dict(Hkv=0), dict(Hkv=8),
               dict(B=-1), dict(T=-1), dict(pages=0), dict(page=24), dict(page=0), dict(page=512), dict(width=0),
               dict(width=1 << 27), dict(H=1 << 26, Hkv=1 << 25, T=1, B=1, page=256), dict(kp=None), dict(vp=0x1008), dict(table=None),
               dict(table=0x1002), dict(ctx=None), dict(ctx=0x1001), dict(tree=0x1004), dict(lse=None), dict(lse=0x1002),
               dict(q=view(2, 4, 3, 64, ptr=0)), dict(o=view(2, 4, 3, 64, strides=(0, 64, 256)))):
        assert attend(lib, **kw) == BAD, kw
    for kw in (dict(d=32), dict(d=256), dict(T=65)):
        assert attend(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(ws=0x1010), dict(ws_bytes=lib.fa_cached_workspace_bytes(2, 4, 2, 3, 64) - 1)):
        assert attend(lib, **kw) == WORKSPACE, kw
    for kw in (dict(B=0), dict(T=0), dict(H=0, Hkv=0)):
        assert attend(lib, kp=None, **kw) == 0, kw


def test_workspace_sizes(lib):
    assert lib.fa_cached_workspace_bytes(2, 4, 2, 65, 64) == 0
    assert lib.fa_cached_workspace_bytes(2, 4, 3, 1, 64) == 0
    assert lib.fa_cached_workspace_bytes(2, 4, 2, 1, 96) == 0
    assert lib.fa_cached_workspace_bytes(1, 1, 1, 1, 128) > 128 * 4
    assert lib.fa_cached_workspace_bytes(8, 64, 1, 64, 128) >= 8 * 64 * 64 * 128 * 4


def append(lib, B=2, Hkv=2, T=3, d=64, pages=10, page=16, width=8, kp=0x1000, table=0x1000, ctx=0x1000, count=None, k=None):
    return lib.fa_cache_append(k or view(B, Hkv, T, d), view(B, Hkv, T, d), kp, 0x1000, table, ctx, count, B, Hkv, T, d,
                               pages, page, width, None)


def compact(lib, B=2, Hkv=2, M=3, d=64, pages=10, page=16, width=8, kp=0x1000, src=0x1000, count=0x1000):
    return lib.fa_cache_compact(kp, 0x1000, 0x1000, 0x1000, src, count, B, Hkv, M, d, pages, page, width, None)


def test_write_arguments(lib):
    for kw in (dict(pages=0), dict(page=8), dict(width=0), dict(kp=None), dict(kp=0x1004), dict(table=None),
               dict(ctx=None), dict(count=0x1002), dict(B=-1), dict(k=view(2, 2, 3, 64, strides=(384, 192, 60)))):
        assert append(lib, **kw) == BAD, kw
    assert append(lib, d=48) == UNSUPPORTED
    assert append(lib, T=1 << 26, Hkv=8) == UNSUPPORTED
    assert append(lib, T=0, kp=None) == 0
    for kw in (dict(src=None), dict(count=None), dict(src=0x1001), dict(pages=-1), dict(page=17), dict(M=-1)):
        assert compact(lib, **kw) == BAD, kw
    for kw in (dict(M=65), dict(d=100)):
        assert compact(lib, **kw) == UNSUPPORTED, kw
    assert compact(lib, M=0, src=None) == 0


def test_python_refuses_what_does_not_fit():
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table, ctx = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.cached_attention(q, pool, pool, table, ctx)
    with pytest.raises(ValueError):
        fa.fa_cache_append(q, q, pool, pool, table, ctx)
    with pytest.raises(ValueError):
        fa.fa_cache_compact(pool, pool, table, ctx, table, ctx)
