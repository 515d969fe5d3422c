"""What the build takes for up to date, and what the binding loads (no GPU)."""

import os
import sysconfig

import pytest
import torch

from bf16_numerics_b200 import _abi, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_library()


@pytest.fixture
def compiled(monkeypatch):
    """Outputs that build_library() would compile, without compiling them."""
    out = []
    monkeypatch.setattr(build, "_compile", lambda cmd, path, verbose: out.append(path))
    return out


def test_a_fresh_build_is_up_to_date(compiled):
    build.build_library()
    assert compiled == []
    build.build_library(force=True)
    assert compiled == [build.LIB_PATH, build.marshal_path()]


@pytest.mark.parametrize("what", ["torch", "python", "abi"])
def test_another_torch_or_python_builds_a_module_of_its_own(compiled, monkeypatch, what):
    """The module holds torch's C++ ABI and Python's C API: one that was built for others is neither up to date nor
    loaded."""
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    elif what == "python":
        monkeypatch.setattr(sysconfig, "get_config_var", lambda name, real=sysconfig.get_config_var:
                            "cpython-999-other" if name == "SOABI" else real(name))
    else:
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    build.build_library()
    assert compiled == [build.marshal_path()]
    monkeypatch.setattr(_abi, "_bound", None)
    with pytest.raises(ImportError, match="missing"):
        _abi.marshal()


@pytest.mark.parametrize("changed,rebuilt", [("fa_torch.cpp", 1), ("fa_cached.cuh", 1), ("fa_b200.h", 2), ("build.py", 2)])
def test_a_newer_source_or_other_flags_rebuild(compiled, monkeypatch, changed, rebuilt):
    real = os.path.getmtime
    monkeypatch.setattr(build.os.path, "getmtime", lambda path: real(path) + (1e9 if path.endswith(changed) else 0))
    build.build_library()
    assert len(compiled) == rebuilt


def test_the_module_that_is_loaded_is_the_running_torchs():
    module = _abi.marshal()
    assert os.path.samefile(module.__file__, build.marshal_path())
    assert torch.__version__ in os.path.basename(module.__file__)
