"""The module for PyTorch is a shortcut: where it does not compile or load, the library
is built and the calls go through ctypes, with a warning."""

import subprocess

import pytest

import ggml_q2_quantized_gb300 as q2k
from ggml_q2_quantized_gb300 import build as q2k_build

torch = pytest.importorskip("torch")


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build folder of its own, its library already there."""
    monkeypatch.setattr(q2k_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(q2k_build, "_build_library", lambda force, verbose: "libq2k.so")
    return tmp_path


def fails(*args, **kw):
    return subprocess.CompletedProcess(args, 1, "", "fatal error: Python.h: No such file or directory")


def missing(*args, **kw):
    raise FileNotFoundError("g++")


@pytest.mark.parametrize("compiler", [fails, missing])
def test_a_module_that_does_not_compile_is_a_warning(elsewhere, monkeypatch, compiler):
    monkeypatch.setattr(q2k_build.subprocess, "run", compiler)
    with pytest.warns(RuntimeWarning, match="ctypes.*(Python.h|g\\+\\+)"):
        assert q2k_build.build() == "libq2k.so"


def test_a_module_of_other_sources_is_not_left(elsewhere, monkeypatch):
    old = elsewhere / f"q2k_torch-{torch.__version__}.so"
    old.write_bytes(b"old")
    monkeypatch.setattr(q2k_build.subprocess, "run", fails)
    with pytest.warns(RuntimeWarning):
        q2k_build.build(force=True)
    assert not old.exists()


def test_a_module_that_does_not_load_is_a_warning(tmp_path, monkeypatch):
    broken = tmp_path / "q2k_torch.so"
    broken.write_bytes(b"not a library")
    q2k_build.build()
    monkeypatch.setattr(q2k, "_quick_mod", None)
    monkeypatch.setattr(q2k._build, "torch_module_path", lambda version: str(broken))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert q2k._quick() is False
    with pytest.raises(TypeError, match="CUDA"):
        q2k.gated_ffn(torch.zeros(1, 256), None, None, 1)
