"""What the build needs: the library nvcc alone, the binding's compiled half
torch and g++ too.  No compiler runs here."""
import importlib.util
import shutil
import subprocess

import pytest

from dynamic_expert_routing_router_b200 import build


@pytest.fixture
def commands(monkeypatch):
    """The commands that the build would run; those of `fails` end with an error."""
    ran, fails = [], []

    def run(cmd, check):
        ran.append(cmd[0].rsplit("/", 1)[-1])
        if ran[-1] in fails:
            raise subprocess.CalledProcessError(1, cmd)
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return ran, fails


def test_everything(commands):
    assert build.build(force=True) == build.LIB
    assert commands[0] == ["nvcc", "g++"]


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_library_needs_neither_torch_nor_a_cpp_compiler(commands, monkeypatch, capsys, missing):
    if missing == "torch":
        found = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else found(n, *a))
        monkeypatch.setattr(build, "build_marshal", lambda *a: pytest.fail("torch was wanted"))
    else:
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n, *a: None if n == "g++" else which(n, *a))
    assert build.build(force=True) == build.LIB
    assert commands[0] == ["nvcc"]
    assert f"{missing} not found" in capsys.readouterr().err


def test_a_failing_cpp_compiler_comes_after_the_library(commands):
    commands[1].append("g++")
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)
    assert commands[0] == ["nvcc", "g++"]
