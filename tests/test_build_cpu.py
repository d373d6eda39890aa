"""What build() compiles and links again, and what it does without torch: the
compilers replaced by recorders, in a folder of the test's own."""
from __future__ import annotations

import os
import types

import pytest

from mamba2_ssm_decode_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build tree whose tools write their output file; `tree.fail` names outputs
    whose tool fails, `tree.made` lists what was made."""
    t = types.SimpleNamespace(made=[], fail=set(), torch=tmp_path / "torch", at=tmp_path)
    t.torch.mkdir()
    (t.torch / "version.py").write_text("__version__ = '1'")
    for name, value in (("BUILD", "_build"), ("LIB", "lib.so"), ("BINDING", "binding.so"),
                        ("STAMP", "_build/stamp")):
        monkeypatch.setattr(b, name, str(tmp_path / value), raising=False)
    monkeypatch.setattr(b, "sources", lambda: [str(tmp_path / "k.cu")])
    (tmp_path / "k.cu").write_text("")
    clock = [os.path.getmtime(b.__file__) + 1e6]

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".so.")[0].removesuffix(".so")
        if name in t.fail:
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no")
        t.made.append(name)
        with open(out, "w"):
            pass
        clock[0] += 10.0    # every file is newer than those made before it
        os.utime(out, (clock[0], clock[0]))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: types.SimpleNamespace(
        submodule_search_locations=[str(t.torch)]) if t.torch else None)
    return t


def test_all_is_built_once(tree):
    assert b.build() == b.LIB
    assert sorted(tree.made) == ["binding", "k.o", "layer_binding.o", "lib"]
    b.build()
    assert len(tree.made) == 4


def test_the_library_is_built_without_torch(tree):
    tree.torch = None
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert sorted(tree.made) == ["k.o", "lib"] and not os.path.exists(b.BINDING)


def test_the_library_is_built_where_the_module_fails(tree):
    tree.fail = {"layer_binding.o"}
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB)


@pytest.mark.parametrize("what", ["binding", "lib"])
def test_a_failed_link_is_made_up_for(tree, what):
    """After a new object file and a link that failed, an old module does not stay."""
    b.build()
    tree.fail, tree.made = {what}, []
    with pytest.raises(RuntimeError, match="link"):
        b.build(force=True)
    tree.fail, tree.made = set(), []
    b.build()
    assert "binding" in tree.made
    tree.made = []
    b.build()
    assert tree.made == []


def test_another_torch_compiles_the_module_again(tree):
    b.build()
    tree.made = []
    (tree.torch / "version.py").write_text("__version__ = '2'")
    b.build()
    assert tree.made == ["layer_binding.o", "binding"]
