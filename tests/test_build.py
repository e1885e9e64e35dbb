"""The in-tree build: the C library does not depend on the module for torch tensors."""

import os
import subprocess
import types

import pytest

from mla_query_projection_gb300 import build


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A build into a folder of its own whose compiler writes empty files."""
    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    for name, file in (("LIB", "libmla_query.so"), ("BUILD", "_build"), ("CALLS", "_tensor_calls.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return tmp_path


def test_builds_both(tree):
    assert build.build() == str(tree / "libmla_query.so")
    assert (tree / "libmla_query.so").exists() and (tree / "_tensor_calls.so").exists()


def test_a_tensor_module_that_fails_leaves_the_library(tree, monkeypatch):
    """It is an error all the same, but one that comes after the link."""
    def fails():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_compile_calls", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert (tree / "libmla_query.so").exists()


def test_without_torch_the_error_says_so(tree, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="torch is not installed"):
        build.build()
    assert (tree / "libmla_query.so").exists() and not (tree / "_tensor_calls.so").exists()


def test_a_library_that_does_not_compile_is_no_library(tree, monkeypatch):
    monkeypatch.setattr(subprocess, "run", lambda *a, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    assert not (tree / "libmla_query.so").exists()
    assert os.path.basename(build.LIB) == "libmla_query.so"
