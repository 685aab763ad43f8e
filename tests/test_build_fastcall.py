"""The compiled argument checks are used only if they were built from the
present sources for the present interpreter and torch; any other file goes."""

import glob
import os
import shutil
import subprocess
import sys
import types

import pytest

from speculative_decoding_tree_03_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build folder and sources of their own, and a compiler that only writes its output."""
    out, inc, csrc = tmp_path / "out", tmp_path / "include", tmp_path / "csrc"
    out.mkdir()
    csrc.mkdir()
    shutil.copytree(b.INCLUDE, inc)
    shutil.copy(os.path.join(b.CSRC, "fastcall.cpp"), csrc)
    monkeypatch.setattr(b, "OUT", str(out))
    monkeypatch.setattr(b, "INCLUDE", str(inc))
    monkeypatch.setattr(b, "CSRC", str(csrc))
    monkeypatch.setattr(b, "FAST", str(out / "_fastcall.so"), raising=False)
    t = types.SimpleNamespace(out=out, header=inc / "specverify.h", rc=0, calls=0)

    def run(cmd, **kw):
        t.calls += 1
        if t.rc == 0:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(str(t.calls))
        return subprocess.CompletedProcess(cmd, t.rc, "", "no compiler")

    monkeypatch.setattr(b.subprocess, "run", run)
    t.files = lambda: sorted(glob.glob(str(out / "_fastcall*")))
    return t


def change_header(t):
    t.header.write_text(t.header.read_text() + "/* another signature */\n")
    os.utime(t.header, (2e9, 2e9))


def test_a_failed_build_leaves_no_stale_module(tree, capsys):
    b._build_fastcall()
    assert len(tree.files()) == 1
    change_header(tree)
    tree.rc = 1
    b._build_fastcall()
    assert tree.files() == [] and "not built" in capsys.readouterr().err


def test_it_is_built_once_and_again_when_something_changes(tree, monkeypatch):
    for _ in range(2):
        b._build_fastcall()
    assert tree.calls == 1
    change_header(tree)
    b._build_fastcall()
    assert tree.calls == 2 and len(tree.files()) == 1
    import torch
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    b._build_fastcall()
    assert tree.calls == 3 and len(tree.files()) == 1
    monkeypatch.setattr(sys.implementation, "cache_tag", "other-1")
    b._build_fastcall()
    assert tree.calls == 4 and len(tree.files()) == 1
    b._build_fastcall(force=True)
    assert tree.calls == 5 and len(tree.files()) == 1


def test_without_torch_the_library_is_built_all_the_same(tree, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch raises ImportError
    b._build_fastcall()
    assert tree.files() == [] and tree.calls == 0 and "not built" in capsys.readouterr().err


def test_a_module_of_other_sources_is_not_loaded(tree, monkeypatch):
    import speculative_decoding_tree_03_gb300 as sv
    b._build_fastcall()
    seen = []
    monkeypatch.setattr("importlib.machinery.ExtensionFileLoader",
                        lambda name, path: seen.append(path) or (_ for _ in ()).throw(ImportError()))
    sv._load_fastcall(None)
    assert seen == tree.files()         # this one would be
    change_header(tree)
    sv._load_fastcall(None)
    assert len(seen) == 1               # no longer
