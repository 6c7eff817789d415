"""What build() makes again, and what it leaves when a part fails: no compiler runs, a stand-in writes the outputs."""
import os
import subprocess
import types

import pytest

from block_sparse_attention_02_gb300 import _abi
from block_sparse_attention_02_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build() on folders of its own; .ran holds the names of the outputs of each command, .fail those that fail."""
    t = types.SimpleNamespace(ran=[], fail=set(), clock=1_000_000_000)
    for name in ("CSRC", "BUILD", "INCLUDE"):
        os.mkdir(tmp_path / name)
        monkeypatch.setattr(b, name, str(tmp_path / name))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmsa.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / os.path.basename(b.BINDING)))

    def touch(path):
        """Writes a file, later than all before it."""
        with open(path, "w") as f:
            f.write("x")
        t.clock += 10
        os.utime(path, (t.clock, t.clock))
    t.touch = touch

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        t.ran.append(name)
        if name in t.fail:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="refused")
        touch(out)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(subprocess, "run", run)
    monkeypatch.setattr(b, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name in ("api.cu", "other.cu", "binding.cpp"):
        touch(os.path.join(b.CSRC, name))
    touch(os.path.join(b.INCLUDE, "msa.h"))

    def built():
        t.ran.clear()
        b.build()
        return sorted(t.ran)
    t.built = built
    t.module, t.library = os.path.basename(b.BINDING), "libmsa.so"
    assert built() == sorted(["api.o", "other.o", "binding.o", t.library, t.module])
    assert built() == []
    return t


def test_what_is_linked_follows_its_objects(tree):
    """A build that ended after an object and before the link leaves the link to the next one."""
    tree.touch(os.path.join(b.BUILD, "binding.o"))
    assert tree.built() == [tree.module]
    tree.touch(os.path.join(b.BUILD, "other.o"))
    assert tree.built() == [tree.library]
    os.remove(b.BINDING)
    assert tree.built() == [tree.module]
    assert tree.built() == []


def test_a_header_reaches_everything(tree):
    tree.touch(os.path.join(b.INCLUDE, "msa.h"))
    assert tree.built() == sorted(["api.o", "other.o", "binding.o", tree.library, tree.module])


def test_another_torch_builds_the_module_again(tree, monkeypatch):
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    assert tree.built() == sorted(["binding.o", tree.module])
    assert tree.built() == []


def test_the_library_is_built_without_the_module(tree):
    """No Python headers: the library is new, no module of the old headers stays beside it, and the build fails."""
    old_name = os.path.join(os.path.dirname(b.BINDING), "_msa_binding.so")
    tree.touch(old_name)
    tree.touch(os.path.join(b.INCLUDE, "msa.h"))
    tree.fail = {"binding.o"}
    before = os.path.getmtime(b.LIB)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.getmtime(b.LIB) > before
    assert not os.path.exists(b.BINDING) and not os.path.exists(old_name)
    tree.fail = set()
    assert tree.built() == sorted(["binding.o", tree.module])


def test_a_failed_link_is_made_up_for(tree):
    tree.touch(os.path.join(b.CSRC, "binding.cpp"))
    tree.fail = {tree.module}
    with pytest.raises(RuntimeError):
        b.build()
    assert not os.path.exists(b.BINDING)
    tree.fail = set()
    assert tree.module in tree.built()


def test_a_module_of_another_torch_is_refused(monkeypatch):
    import torch
    b.build()
    _abi.binding()
    monkeypatch.setattr(_abi, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    with pytest.raises(RuntimeError, match="9.9.9"):
        _abi.binding()
