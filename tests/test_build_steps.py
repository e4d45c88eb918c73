"""The library and the binding's extension are built one after the other (CPU only; the
compilers are replaced by a writer of empty files)."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from bit_quantized_matmul_amd import build


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """Compilers that write their output, or fail where `fails` names the source; the commands."""
    state = {"fails": "", "commands": []}

    def run(cmd, **kw):
        state["commands"].append(cmd)
        if state["fails"] and any(str(c).endswith(state["fails"]) for c in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "refused")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(" ".join(map(str, cmd)))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libbqm.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    return state


def test_library_and_extension(steps):
    assert build.build(verbose=False) == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.CALLS)


def test_library_without_pytorch(steps, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)              # import torch raises ImportError
    assert build.build(verbose=False) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
    assert "PyTorch" in capsys.readouterr().err


def test_library_where_the_extension_does_not_compile(steps):
    steps["fails"] = "calls.cpp"
    with pytest.raises(RuntimeError, match="calls.cpp"):
        build.build(verbose=False)
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_extension_of_an_older_library_does_not_stay(steps, monkeypatch):
    """What is left of an earlier build would call the new library by the old declarations."""
    build.build(verbose=False)
    steps["fails"] = "calls.cpp"
    with pytest.raises(RuntimeError):
        build.build(verbose=False)
    assert not os.path.exists(build.CALLS)
    steps["fails"] = ""
    build.build(verbose=False)
    monkeypatch.setitem(sys.modules, "torch", None)
    build.build(verbose=False)
    assert not os.path.exists(build.CALLS)


def test_no_extension_without_a_library(steps):
    steps["fails"] = "moe.hip"
    with pytest.raises(RuntimeError, match="moe.hip"):
        build.build(verbose=False)
    assert not os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
