"""The build on a machine that lacks what the compiled Python calls need: the C library, which needs neither Python's nor
PyTorch's headers, is built all the same, and no stale module is left in the calls' place."""
import os
import sys

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    from sequential_rnn_gb300 import build
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    for name in ("LIB", "LIB_BC", "BINDING"):
        monkeypatch.setattr(build, name, str(tmp_path / (name + ".so")))
    monkeypatch.setattr(build, "SOURCES", ["linattn_plan.cu"])  # one small translation unit stands for all
    with open(build.BINDING, "w") as f:
        f.write("made from an older source")
    os.utime(build.BINDING, (0, 0))
    return build


@pytest.mark.parametrize("lacking", ["a compiler that suits the headers", "a compiler", "torch"])
def test_the_library_is_built_without_the_python_calls(build, monkeypatch, lacking):
    if lacking == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setenv("CXX", "false" if "suits" in lacking else "/nonexistent/c++")
    with pytest.warns(RuntimeWarning, match="_binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_the_bounds_check_build_has_no_python_calls(build, monkeypatch):
    def no(*a, **k):
        raise AssertionError("the Python calls are the normal build's")
    monkeypatch.setattr(build, "binding", no)
    assert build.build(bounds_check=True) == build.LIB_BC and os.path.exists(build.LIB_BC)


def test_a_kernel_that_does_not_compile_fails_the_build(build, monkeypatch):
    monkeypatch.setattr(build, "ARCH", ["-gencode", "arch=compute_0,code=sm_0"])
    monkeypatch.setattr(build, "binding", lambda *a, **k: (None, lambda: None))
    with pytest.raises(RuntimeError, match="linattn_plan.cu"):
        build.build()
    assert not os.path.exists(build.LIB)
