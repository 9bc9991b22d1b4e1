"""The build's parts: libee.so comes without PyTorch and whatever becomes of the binding, and
the binding is rebuilt when what it was built with changes.  CPU only; a one-function
library stands in for the kernels."""
import ctypes
import os
import sys

import pytest

import early_exit_decoding_layer_gb300 as ee
from early_exit_decoding_layer_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A tree of one .cu file and a binding source without PyTorch in it."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (csrc / "bind.cpp").write_text('extern "C" int one(); extern "C" int two() { return 2 * one(); }\n')
    for name, value in dict(HERE=tmp_path, CSRC=csrc, BUILD=tmp_path / "_build", LIB=tmp_path / "libee.so",
                            BINDING=tmp_path / "_binding.so", BINDING_SRC=csrc / "bind.cpp").items():
        monkeypatch.setattr(build, name, str(value))
    return tmp_path


def library(small):
    return ctypes.CDLL(str(small / "libee.so"))


def test_library_builds_without_pytorch(small, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build() == str(small / "libee.so")
    assert library(small).one() == 1 and not (small / "_binding.so").exists()


@pytest.mark.parametrize("cxx", ["false", "/no/such/compiler"])
def test_a_failed_binding_leaves_the_library(small, monkeypatch, capfd, cxx):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", cxx)
    assert build.build() == str(small / "libee.so")
    assert library(small).one() == 1 and not (small / "_binding.so").exists()
    assert "binding to PyTorch was not built" in capfd.readouterr().err
    monkeypatch.delenv("CXX")   # tried again in the next build
    build.build()
    assert (small / "_binding.so").exists()


def test_a_failed_library_is_an_error(small):
    (small / "csrc" / "one.cu").write_text("#error no\n")
    with pytest.raises(RuntimeError):
        build.build()


def test_binding_follows_pytorch_python_and_commands(small, monkeypatch):
    pytest.importorskip("torch")
    runs = []
    run = build._run
    monkeypatch.setattr(build, "_run", lambda cmd: (runs.append(cmd), run(cmd))[1])
    compiles = lambda: sum(build.BINDING_SRC in c for c in runs)  # noqa: E731
    build.build()
    build.build()
    assert compiles() == 1 and (small / "_binding.so").exists()
    text = build._torch_version(build.torch_dir())
    monkeypatch.setattr(build, "_torch_version", lambda t: text + "\ngit_version = 'other'\n")
    build.build()
    build.build()
    assert compiles() == 2
    monkeypatch.setattr(build.sys, "version", "another Python")
    build.build()
    assert compiles() == 3
    lib = os.path.getmtime(small / "libee.so")
    os.remove(small / "_binding.so")
    build.build()
    assert compiles() == 4 and (small / "_binding.so").exists() and os.path.getmtime(small / "libee.so") == lib


def test_binding_is_of_this_python_and_pytorch(monkeypatch):
    torch = pytest.importorskip("torch")
    build.build()
    native = ee._cache_ops()
    assert native.torch_version == torch.__version__
    assert sys.implementation.cache_tag.split("-")[1] in os.path.basename(native.__file__)
    monkeypatch.setattr(ee, "_native", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(RuntimeError, match="built for PyTorch"):
        ee._cache_ops()
