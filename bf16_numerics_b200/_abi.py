"""ctypes view of libfa_b200.so (include/fa_b200.h).  Argument marshalling only.

The library must exist in-tree (``python -m bf16_numerics_b200.build``);
there is no fallback of any kind: a missing or unloadable library raises.
"""

from __future__ import annotations

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa_b200.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_WORKSPACE = 3
FA_ERR_CUDA = 4
FA_ERR_TIMEOUT = 5
FA_ERR_BAD_PAGE = 6

FA_SOFTMAX_STANDARD = 0
FA_SOFTMAX_STABILIZED = 1
FA_SOFTMAX_STABILIZED_MARGIN = 2

FA_KERNEL_FWD = 0
FA_KERNEL_BWD_DELTA = 1
FA_KERNEL_BWD_MAIN = 2
FA_KERNEL_BWD_DQ = 3
FA_NUM_KERNELS = 4

# kernel ids in the device error word (fa_device_error) and for fa_debug_inject_stall
FA_ERRWORD_FWD = 1
FA_ERRWORD_BWD_D64 = 3
FA_ERRWORD_BWD_D128 = 4
FA_ERRWORD_CACHE_PAGE = 6
FA_ERRWORD_CACHED = 7
KERNEL_NAMES = ("fa_fwd_kernel", "fa_bwd_delta_kernel", "fa_bwd_main_kernel", "fa_bwd_dq_convert_kernel")

# every symbol include/fa_b200.h declares
EXPORTS = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_bwd_workspace_delta_offset",
           "fa_bwd_workspace_dq_offset", "fa_status_string", "fa_device_error", "fa_timing_enable",
           "fa_timing_read", "fa_bwd_noalloc", "fa_last_error_string", "fa_fwd_o_hp", "fa_bwd_o_hp",
           "fa_debug_set_wait_limit_ns", "fa_debug_inject_stall", "fa_window_fwd", "fa_window_bwd",
           "fa_window_bwd_workspace_bytes", "fa_cached_workspace_bytes", "fa_cached_fwd", "fa_cache_append",
           "fa_cache_compact")


class FaRowStats(ctypes.Structure):
    _fields_ = [("rm", ctypes.c_void_p), ("rs", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("pbar_max", ctypes.c_void_p)]


class FaView(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_n", ctypes.c_longlong)]


_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bf16_numerics_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, ctypes.POINTER(FaRowStats), i, i, i, i, i, i, f, vp]
    lib.fa_fwd.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, i, f, vp]
    lib.fa_bwd.restype = i
    lib.fa_fwd_o_hp.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.POINTER(FaRowStats), i, i, i, i, i, i, f, vp]
    lib.fa_fwd_o_hp.restype = i
    lib.fa_bwd_o_hp.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, i, f, vp]
    lib.fa_bwd_o_hp.restype = i
    for name in ("fa_bwd_workspace_bytes", "fa_bwd_workspace_delta_offset", "fa_bwd_workspace_dq_offset"):
        getattr(lib, name).argtypes = [i, i, i, i]
        getattr(lib, name).restype = sz
    view = ctypes.POINTER(FaView)
    lib.fa_window_fwd.argtypes = [view] * 4 + [vp, ctypes.POINTER(FaRowStats)] + [i] * 8 + [f, vp]
    lib.fa_window_fwd.restype = i
    lib.fa_window_bwd.argtypes = [view] * 5 + [vp, vp] + [view] * 3 + [vp, sz] + [i] * 8 + [f, vp]
    lib.fa_window_bwd.restype = i
    lib.fa_window_bwd_workspace_bytes.argtypes = [i] * 7
    lib.fa_window_bwd_workspace_bytes.restype = sz
    lib.fa_cached_workspace_bytes.argtypes = [i] * 5
    lib.fa_cached_workspace_bytes.restype = sz
    lib.fa_cached_fwd.argtypes = [view] + [vp] * 5 + [view, vp, vp, sz] + [i] * 11 + [f, vp]
    lib.fa_cached_fwd.restype = i
    lib.fa_cache_append.argtypes = [view, view] + [vp] * 5 + [i] * 7 + [vp]
    lib.fa_cache_append.restype = i
    lib.fa_cache_compact.argtypes = [vp] * 6 + [i] * 7 + [vp]
    lib.fa_cache_compact.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_last_error_string.argtypes = []
    lib.fa_last_error_string.restype = ctypes.c_char_p
    lib.fa_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
    lib.fa_device_error.restype = i
    lib.fa_debug_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.fa_debug_set_wait_limit_ns.restype = i
    lib.fa_debug_inject_stall.argtypes = [ctypes.c_uint]
    lib.fa_debug_inject_stall.restype = i
    lib.fa_timing_enable.argtypes = [i]
    lib.fa_timing_enable.restype = i
    lib.fa_timing_read.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_double)]
    lib.fa_timing_read.restype = i
    _lib = lib
    return lib


#: entry points that csrc/fa_torch.cpp calls, in its order
MARSHALLED = ("fa_window_fwd", "fa_window_bwd", "fa_window_bwd_workspace_bytes", "fa_cached_fwd",
              "fa_cached_workspace_bytes", "fa_cache_append", "fa_cache_compact")
_bound = None


def marshal():
    """The C++ marshalling module of this Python and torch, bound to the loaded library."""
    global _bound
    if _bound is None:
        import importlib.util

        from .build import marshal_path

        lib, path = load(), marshal_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python -m bf16_numerics_b200.build`")
        spec = importlib.util.spec_from_file_location(f"{__package__}._marshal", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in MARSHALLED))
        _bound = module
    return _bound


def status_string(code: int) -> str:
    return load().fa_status_string(code).decode()
