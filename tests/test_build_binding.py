"""The binding belongs to the PyTorch and interpreter that it was compiled against: after a change of either an older
file, however new its time, is neither kept by the build nor loaded."""
import os

import pytest
import torch

import differential_latent_attention_b200 as gdla
from differential_latent_attention_b200 import _build, ops


def test_a_binding_of_another_pytorch_is_not_taken(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    commands = []

    def compile_to(cmd):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(_build, "_compile", compile_to)
    first = _build.build_binding()
    assert os.path.exists(first) and len(commands) == 1
    assert _build.build_binding() == first and len(commands) == 1       # nothing has changed
    later = os.path.getmtime(first) + 1000
    os.utime(first, (later, later))
    monkeypatch.setattr(torch, "__version__", "99.0.0+cu000")
    second = _build.build_binding()
    assert second != first and len(commands) == 2 and os.path.exists(second)
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: ".other-interpreter.so")
    assert _build.build_binding() not in (first, second) and len(commands) == 3
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    _build.build_binding()
    assert len(commands) == 4


def test_a_binding_of_another_pytorch_is_not_loaded(monkeypatch):
    _build.build()
    monkeypatch.setattr(ops, "_native", None)
    monkeypatch.setattr(torch, "__version__", "99.0.0+cu000")
    with pytest.raises(RuntimeError, match="build it with"):
        gdla.cache_append(None, None, None, None, None, None, None, None)
