"""The native helpers are rebuilt for another torch or interpreter, and refuse to run with one
that they were not built for."""
import os
import time

import pytest
import torch

from scaling_aware_transpose_b200 import build, moe


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A finished build of the binding elsewhere, its compiler replaced by a counter."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").write("built")
        return type("R", (), dict(returncode=0, stdout="", stderr=""))

    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_moe_binding.so"))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "key"))
    monkeypatch.setattr(build.subprocess, "run", run)
    build._build_binding(False)
    os.utime(build.BINDING, (time.time() + 60,) * 2)
    assert len(calls) == 1
    return calls


def test_a_finished_binding_is_kept(tree):
    build._build_binding(False)
    assert len(tree) == 1
    build._build_binding(True)
    assert len(tree) == 2


@pytest.mark.parametrize("what", ["torch", "abi", "python"])
def test_another_torch_or_interpreter_rebuilds(tree, monkeypatch, what):
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    else:
        import sysconfig
        real = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda k: "other" if k == "SOABI" else real(k))
    build._build_binding(False)
    assert len(tree) == 2
    os.utime(build.BINDING, (time.time() + 60,) * 2)
    build._build_binding(False)
    assert len(tree) == 2


def test_a_binding_without_its_key_is_rebuilt(tree):
    os.remove(build.BINDING_KEY)
    build._build_binding(False)
    assert len(tree) == 2


def test_a_binding_of_another_torch_is_refused(monkeypatch):
    build.build()
    monkeypatch.setattr(moe, "_native", None)
    moe._binding()
    monkeypatch.setattr(moe, "_native", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    with pytest.raises(RuntimeError, match="built for torch"):
        moe._binding()
