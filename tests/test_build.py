"""The build's order and what it links again, with stand-ins for the compilers."""

import os
import subprocess
import types

import pytest
import torch

from quantization_aware_attention_gb300 import build as qbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An empty build tree; every command makes its output and is recorded."""
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(qbuild, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(qbuild, "LIB_PATH", str(tmp_path / "libqat_attn.so"))
    monkeypatch.setattr(qbuild, "EXT_PATH", str(tmp_path / "_qat_torch.so"))
    monkeypatch.setattr(qbuild, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(subprocess, "run", run)
    return commands


def _ext_links(commands):
    """The objects that the extension was linked from, in order."""
    return [c[2] for c in commands if "-shared" in c and "-ltorch" in c]


def test_the_library_is_linked_even_if_the_extension_fails(tree, monkeypatch):
    def fails(verbose):
        raise RuntimeError("no compiler")

    monkeypatch.setattr(qbuild, "_compile_ext", fails)
    with pytest.raises(RuntimeError, match="no compiler"):
        qbuild.build()
    assert os.path.exists(qbuild.LIB_PATH)


def test_without_torch_the_library_is_built_alone(tree, monkeypatch):
    find = qbuild.importlib.util.find_spec
    monkeypatch.setattr(qbuild.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert qbuild.build() == qbuild.LIB_PATH and os.path.exists(qbuild.LIB_PATH)
    assert not os.path.exists(qbuild.EXT_PATH) and not _ext_links(tree)


def test_the_extension_is_linked_again_for_another_torch(tree, monkeypatch):
    """There and back: the first torch's object is older than the extension of the second."""
    for version in ("9.0", "9.0", "9.1", "9.0"):
        monkeypatch.setattr(torch, "__version__", version)
        qbuild.build()
    links = _ext_links(tree)
    assert len(links) == 3 and links[0] == links[2] != links[1]
    monkeypatch.setattr(torch, "__file__", "/elsewhere/torch/__init__.py")  # the same version in another place
    qbuild.build()
    links = _ext_links(tree)
    assert len(links) == 4 and links[3] != links[2] and any("/elsewhere/torch/lib" in a for a in tree[-1])


def test_nothing_is_built_twice(tree):
    qbuild.build()
    n = len(tree)
    qbuild.build()
    assert len(tree) == n
