"""What the build needs: the library nvcc alone, the binding's compiled half
torch and g++ too.  No compiler runs here."""
import importlib.util
import os
import shutil
import subprocess

import pytest
import torch

from dynamic_expert_routing_router_b200 import abi, build


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


def test_the_binding_belongs_to_one_torch(commands, monkeypatch, tmp_path):
    """Another torch: the module of the one before is neither kept nor loaded."""
    assert os.path.exists(build.marshal_path())
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    first = build.marshal_path()
    for name in (os.path.basename(first), "_marshal.so"):
        (tmp_path / name).write_bytes(b"")
        os.utime(tmp_path / name, (2e9, 2e9))  # newer than its source
    assert build.build_marshal() == first and commands[0] == []
    monkeypatch.setattr(torch, "__version__", "99.0")
    monkeypatch.setattr(abi, "_marshal_module", None)
    with pytest.raises(RuntimeError, match="99.0.*build it"):
        abi._marshal()
    assert build.build_marshal() == build.marshal_path() != first and commands[0] == ["g++"]
    assert os.listdir(tmp_path) == []  # the old ones are gone (and no compiler ran here)
