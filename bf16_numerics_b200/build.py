"""Build libfa_b200.so in-tree with nvcc (sm_100a only).

    python -m bf16_numerics_b200.build [--force] [--verbose]

The library is a single translation unit (csrc/fa_lib.cu) that includes the
kernel headers; the CUDA runtime is linked statically so the library does not
depend on the runtime version PyTorch ships.  The marshalling module
(csrc/fa_torch.cpp, g++) turns torch tensors into calls of the library; it is
bound to the C++ ABI of one torch and the C API of one Python, which its file
name therefore carries: another torch in the same tree finds none of its own
and builds one.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libfa_b200.so")
SOURCES = [os.path.join(CSRC, "fa_lib.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(INCLUDE, "fa_b200.h"), os.path.abspath(__file__)]

MARSHAL_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
MARSHAL_DEPS = [MARSHAL_SOURCE, os.path.join(INCLUDE, "fa_b200.h"), os.path.abspath(__file__)]


def marshal_path() -> str:
    """The marshalling module of the running Python and torch."""
    import sysconfig

    import torch

    abi = f"{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(PKG_DIR, f"_marshal.{abi}.so")


def marshal_command(out: str) -> list[str]:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import CUDA_HOME, include_paths, library_paths

    libs = library_paths()
    cuda = os.path.join(CUDA_HOME or os.path.dirname(os.path.dirname(nvcc_path())), "include")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
            *(f"-I{d}" for d in include_paths()), f"-I{cuda}", f"-I{sysconfig.get_paths()['include']}", MARSHAL_SOURCE,
            "-o", out, *(f"-L{d}" for d in libs), *(f"-Wl,-rpath,{d}" for d in libs), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python"]


def nvcc_path() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")
    return cand


def nvcc_command(out: str = LIB_PATH, extra=()) -> list[str]:
    return [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
            "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", f"-I{INCLUDE}", *extra, "-o", out, *SOURCES]


def up_to_date(out: str = LIB_PATH, deps=DEPS) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(p) <= t for p in deps)


def _compile(cmd: list[str], out: str, verbose: bool) -> None:
    tmp = out + ".tmp"
    cmd = [tmp if arg == out else arg for arg in cmd]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed with exit code {res.returncode}")
    os.replace(tmp, out)


def build_library(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        _compile(nvcc_command(extra=("-Xptxas", "-v") if verbose else ()), LIB_PATH, verbose)
    marshal = marshal_path()
    if force or not up_to_date(marshal, MARSHAL_DEPS):
        _compile(marshal_command(marshal), marshal, verbose)
    return LIB_PATH


if __name__ == "__main__":
    build_library(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB_PATH)
