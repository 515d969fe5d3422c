"""What fa_window_fwd / fa_window_bwd and their Python forms refuse (no GPU: refused before anything is launched)."""

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
    st = strides or (H * N * d, N * d, d)
    return _abi.FaView(ptr, *st)


def call(lib, name, B=2, H=4, Hkv=2, N=300, d=64, window=64, sinks=4, mode=1, beta=2.0, lse=0x1000, row_m=0x1000,
         ws=0x100000, ws_bytes=1 << 40, **views):
    q = lambda n: ctypes.byref(views[n]) if n in views else ctypes.byref(view(B, H, N, d))
    kv = lambda n: ctypes.byref(views[n]) if n in views else ctypes.byref(view(B, Hkv, N, d))
    tail = (B, H, Hkv, N, d, window, sinks, mode, beta, None)
    if name == "fwd":
        return lib.fa_window_fwd(q("q"), kv("k"), kv("v"), q("o"), lse, None, *tail)
    return lib.fa_window_bwd(q("q"), kv("k"), kv("v"), q("o"), q("dO"), lse, row_m, q("dq"), kv("dk"), kv("dv"), ws,
                             ws_bytes, *tail)


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_sizes_and_modes(lib, name):
    for kw in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(mode=3), dict(mode=-1), dict(beta=1.0),
               dict(beta=float("nan")), dict(Hkv=3), dict(Hkv=0), dict(Hkv=8), dict(Hkv=-1), dict(B=-1), dict(N=-1),
               dict(H=-4), dict(lse=None), dict(lse=0x1002), dict(B=1 << 20, H=1 << 10, N=1 << 12)):
        assert call(lib, name, **kw) == BAD, kw
    for d in (0, 32, 96, 256):
        assert call(lib, name, d=d) == UNSUPPORTED
    for kw in (dict(B=0), dict(N=0), dict(H=0, Hkv=0)):  # nothing to do: no pointer is looked at
        assert call(lib, name, lse=None, **kw) == 0


@pytest.mark.parametrize("name,n", [("fwd", "q"), ("fwd", "o"), ("fwd", "k"), ("bwd", "dO"), ("bwd", "dk"), ("bwd", "dq")])
def test_views(lib, name, n):
    B, H, N, d = 2, 2 if n in ("k", "dk") else 4, 300, 64
    good = (H * N * d, N * d, d)
    for strides in ((0, good[1], good[2]), (good[0], 0, good[2]), (good[0], good[1], 0), (good[0], good[1], -d),
                    (good[0], good[1], d + 4), (good[0], good[1], d - 8), (good[0], (N - 1) * d, d),
                    (good[0] - 8, good[1], d), (1 << 39, good[1], d)):
        assert call(lib, name, **{n: view(B, H, N, d, strides=strides)}) == BAD, strides
    assert call(lib, name, **{n: view(B, H, N, d, ptr=0)}) == BAD
    assert call(lib, name, **{n: view(B, H, N, d, ptr=0x100008)}) == BAD


def test_workspace(lib):
    need = lib.fa_window_bwd_workspace_bytes(2, 4, 2, 300, 64, 64, 4)
    assert need >= 2 * 4 * 300 * (64 + 1) * 4
    assert call(lib, "bwd", ws=None) == WORKSPACE
    assert call(lib, "bwd", ws=0x100080) == WORKSPACE
    assert call(lib, "bwd", ws_bytes=need - 1) == WORKSPACE
    assert call(lib, "bwd", row_m=None) == BAD
    assert lib.fa_window_bwd_workspace_bytes(2, 4, 3, 300, 64, 64, 4) == 0
    assert lib.fa_window_bwd_workspace_bytes(2, 4, 2, 300, 80, 64, 4) == 0
    assert lib.fa_window_bwd_workspace_bytes(2, 4, 2, 300, 64, 0, 4) == 0


def test_python_refuses_host_tensors():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.window_attention_forward(x, x, x, 4)
    with pytest.raises(TypeError):
        fa.window_attention_forward(None, x, x, 4)


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (2**31, 0), (2**32 + 5, 0), (4, -1), (4, 2**31)])
def test_python_refuses_masks_that_do_not_fit(window, sinks):
    with pytest.raises(ValueError):
        fa.fa_window_bwd_workspace_bytes(1, 2, 2, 100, 64, window, sinks)
