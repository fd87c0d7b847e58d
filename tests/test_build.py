"""What build() does where torch, its headers or its version are not what they were; no compiler is run (no GPU needed)."""
import os
import subprocess
import sys

import pytest

from state_space_sequence_ssd_gb300 import build as B


@pytest.fixture
def made(tmp_path, monkeypatch):
    """build() into an empty folder, its compilers replaced by ones that note the output; `made.fails` names one that fails."""
    class Made(list):
        fails = None

    outputs = Made()

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        outputs.append(name)
        if name == outputs.fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libssd_gb300.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "ssd_layer_binding.so"))
    return outputs


def test_both_are_built_once(made):
    assert B.build() == B.LIB and os.path.exists(B.LIB) and os.path.exists(B.BINDING)
    n = len(made)
    B.build()
    assert len(made) == n, "nothing is stale"


def test_the_library_needs_no_torch(made, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    with pytest.warns(UserWarning, match="torch"):
        assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_the_library_is_there_when_the_binding_does_not_compile(made):
    made.fails = "layer_binding.o"
    with pytest.raises(RuntimeError, match="no such header"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_another_torch_makes_the_binding_stale(made, monkeypatch, tmp_path):
    B.build()
    import torch
    other = tmp_path / "torch"
    os.makedirs(other / "include" / "ATen")
    (other / "include" / "ATen" / "ATen.h").write_text("")
    (other / "version.py").write_text("__version__ = '0.0.1'\n")
    (other / "__init__.py").write_text("")
    n = len(made)
    monkeypatch.setattr(torch, "__file__", str(other / "__init__.py"))
    monkeypatch.setattr(torch.__spec__, "origin", str(other / "__init__.py"))
    B.build()
    assert made[n:] == ["layer_binding.o", "ssd_layer_binding.so"]
