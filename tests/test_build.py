"""What the build needs and when it compiles again (no GPU; nvcc is stood in for)."""

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "sub_bit_sparse_b200"


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources, and an nvcc that only leaves its output file."""
    shutil.copytree(os.path.join(ROOT, PKG), tmp_path / PKG,
                    ignore=shutil.ignore_patterns("*.so", "_build", "__pycache__"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text('#!/bin/sh\nwhile [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n')
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    return tmp_path


def _module(tree):
    spec = importlib.util.spec_from_file_location("build_of_a_copy", tree / PKG / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_library_builds_without_torch(tree):
    code = f"""
import importlib.abc, importlib.util, sys
class NoTorch(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named " + repr(name), name=name)
sys.meta_path.insert(0, NoTorch())
find = importlib.util.find_spec
importlib.util.find_spec = lambda name, package=None: None if name == "torch" else find(name, package)
spec = importlib.util.spec_from_file_location("b", {str(tree / PKG / "build.py")!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
print(b.build(), b.build(debug=True))
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    assert (tree / PKG / "libstq1.so").exists() and (tree / PKG / "libstq1_debug.so").exists()
    assert not (tree / PKG / "_dense_calls.so").exists()


def test_library_is_there_when_the_binding_cannot_be_built(tree, monkeypatch):
    pytest.importorskip("torch")
    b = _module(tree)
    (tree / PKG / "binding" / "dense_calls.cpp").write_text("#error no headers")
    with pytest.raises(RuntimeError, match="dense_calls"):
        b.build()
    assert (tree / PKG / "libstq1.so").exists()


def test_binding_is_compiled_again_for_another_torch(tree, monkeypatch):
    pytest.importorskip("torch")
    b = _module(tree)
    runs = []

    def run(cmd, verbose):
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    b.build_binding()
    b.build_binding()
    assert len(runs) == 1                                   # up to date
    b.build_binding(force=True)
    assert len(runs) == 2
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda n: "99.0" if n == "torch" else real(n))
    b.build_binding()
    assert len(runs) == 3
    b.build_binding()
    assert len(runs) == 3
