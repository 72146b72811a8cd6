"""build.py: the library is compiled first and without torch; the native module again when its sources
or torch's version change. No compiler runs here: commands are recorded and make empty files."""
import os
import sys

import pytest

from expert_routing_grouped_layer_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs in a folder of their own; the commands that it runs."""
    ran = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        ran.append("library" if "libmoe.so" in out else "binding")
        open(out, "w").close()
    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(B, "BINDING_STAMP", str(tmp_path / "_binding.torch"))
    return ran


def test_library_first_then_nothing_to_do(tree):
    B.build()
    assert tree == ["library", "binding"]
    B.build()
    assert tree == ["library", "binding"]
    B.build(force=True)
    assert tree == ["library", "binding"] * 2


def test_library_without_torch(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert B.build() == B.LIB and tree == ["library"] and os.path.exists(B.LIB)
    assert "_binding.so is not built" in capsys.readouterr().err


def test_library_is_there_when_the_module_fails(tree, monkeypatch):
    run = B.subprocess.run

    def failing(cmd, check):
        if cmd[0] == "g++":
            raise B.subprocess.CalledProcessError(1, cmd)
        run(cmd, check)
    monkeypatch.setattr(B.subprocess, "run", failing)
    with pytest.raises(B.subprocess.CalledProcessError):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_module_follows_torch_and_its_sources(tree, monkeypatch):
    import torch
    B.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    B.build()
    assert tree == ["library", "binding", "binding"]
    B.build()
    assert len(tree) == 3
    t = os.path.getmtime(B.BINDING_SRC) - 10
    os.utime(B.BINDING, (t, t))
    B.build()
    assert tree[3:] == ["binding"]
