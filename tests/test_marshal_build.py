"""The module of the paged calls' host work is compiled against one torch, one Python and one C header: a file made
for others is never loaded, and a build that fails leaves none."""
import os
import shutil

import pytest
import torch

from token_tree_verification_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of what the module is made of, with files that an earlier version left."""
    here = tmp_path / "package"
    shutil.copytree(build.CSRC, here / "csrc")
    shutil.copytree(os.path.join(os.path.dirname(build.HERE), "include"), tmp_path / "include")
    monkeypatch.setattr(build, "HERE", str(here))
    monkeypatch.setattr(build, "CSRC", str(here / "csrc"))
    for name in ("_marshal.so", "_marshal_0123456789abcdef.so"):
        (here / name).write_bytes(b"compiled against something else")
    return here


def change_torch(tree, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "1.2.3")


def change_torch_commit(tree, monkeypatch):
    monkeypatch.setattr(torch.version, "git_version", "0" * 40)


def change_python(tree, monkeypatch):
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-313")


def change_header(tree, monkeypatch):
    path = tree.parent / "include" / "spec_tree.h"
    path.write_text(path.read_text() + "/* a changed signature */\n")
    os.utime(path, (0, 0))      # older than every file


def change_source(tree, monkeypatch):
    path = tree / "csrc" / "marshal.cpp"
    path.write_text(path.read_text() + "// changed\n")
    os.utime(path, (0, 0))


@pytest.mark.parametrize("change", [change_torch, change_torch_commit, change_python, change_header, change_source])
def test_the_file_is_named_after_what_it_was_compiled_against(tree, monkeypatch, change):
    before = build.marshal_path()
    assert os.path.dirname(before) == str(tree) and build.marshal_path() == before
    change(tree, monkeypatch)
    assert build.marshal_path() != before


def test_a_build_that_fails_leaves_no_module(tree, monkeypatch, capsys):
    monkeypatch.setenv("CXX", shutil.which("false"))
    assert not build.build_marshal()
    assert "not built" in capsys.readouterr().err
    assert [f for f in os.listdir(tree) if f.startswith("_marshal")] == []


def test_a_build_that_is_forced_and_fails_leaves_no_module(tree, monkeypatch):
    monkeypatch.setenv("CXX", shutil.which("false"))
    with open(build.marshal_path(), "wb") as f:
        f.write(b"of the right name")
    assert build.build_marshal() and os.listdir(tree).count(os.path.basename(build.marshal_path())) == 1
    assert not build.build_marshal(force=True)
    assert [f for f in os.listdir(tree) if f.startswith("_marshal")] == []


def test_only_the_module_of_the_right_name_is_loaded(lib, tree, monkeypatch):
    assert build.build_marshal()
    kept = binding._marshal
    try:
        binding._load_marshal(lib)
        assert binding._marshal is not None
        good = build.marshal_path()
        monkeypatch.setattr(torch, "__version__", "1.2.3")
        binding._load_marshal(lib)      # what is there was compiled against another torch
        assert binding._marshal is None
        shutil.copy(good, tree / "_marshal.so")
        binding._load_marshal(lib)
        assert binding._marshal is None
        with open(build.marshal_path(), "wb") as f:
            f.write(b"no module")
        binding._load_marshal(lib)
        assert binding._marshal is None
    finally:
        binding._marshal = kept
