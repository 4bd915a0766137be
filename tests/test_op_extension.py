"""The operators without their extension module: a missing one, one for another torch, one that does
not build.  Calls then run through the Python code and the library alone."""
import os
import subprocess
import sys
import types

import pytest
import torch

import mixture_experts_layer_mok_amd as package
from mixture_experts_layer_mok_amd import _lib as L
from mixture_experts_layer_mok_amd import build, ops

NAME = package.__name__ + "._fast"


def _hide(monkeypatch, module):
    monkeypatch.delattr(package, "_fast", raising=False)
    monkeypatch.setitem(sys.modules, NAME, module)
    monkeypatch.setattr(ops, "_fast", None)
    monkeypatch.setattr(ops, "_bound", False, raising=False)


def _empty_call():
    ops._call("mok_permute", 0, None, 64, None, 0, 2, 64, None, 64, 0, None)


def test_a_missing_module(monkeypatch):
    _hide(monkeypatch, None)
    with pytest.warns(RuntimeWarning, match="_fast is not used"):
        _empty_call()
    assert ops._fast is None
    with pytest.raises(L.MokError):  # looked for once; the library's own refusals as ever
        ops._call("mok_permute", 9, None, 64, None, 0, 2, 64, None, 64, 0, None)


def test_a_module_for_another_torch(monkeypatch):
    other = types.ModuleType(NAME)
    other.torch_version = "0.0"
    other.bind = lambda *a: pytest.fail("bound")
    _hide(monkeypatch, other)
    monkeypatch.setattr(package, "_fast", other, raising=False)
    with pytest.warns(RuntimeWarning, match="built for torch 0.0"):
        _empty_call()
    assert ops._fast is None


def test_the_built_module_fits(monkeypatch):
    from mixture_experts_layer_mok_amd import _fast

    assert _fast.torch_version == torch.__version__
    monkeypatch.setattr(ops, "_fast", None)
    monkeypatch.setattr(ops, "_bound", False)
    _empty_call()
    assert ops._fast is _fast


def test_a_build_without_a_host_compiler(monkeypatch, tmp_path, capfd):
    """The library does not need it; what an earlier build left is not taken for the new module."""
    old = tmp_path / "_fast.so"
    old.write_bytes(b"old")
    run = subprocess.run

    def no_gpp(cmd, *a, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return run(cmd, *a, **kw)

    monkeypatch.setattr(build, "FAST", str(old))
    monkeypatch.setattr(build, "OUT", str(tmp_path / "libmok.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "sources", lambda: [os.path.join(build.CSRC, "api.hip")])
    monkeypatch.setattr(subprocess, "run", no_gpp)
    assert build.build(verbose=False) == str(tmp_path / "libmok.so")
    assert os.path.exists(tmp_path / "libmok.so") and not old.exists()
    assert "_fast.so is not built" in capfd.readouterr().err
