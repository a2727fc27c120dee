"""What build_library() compiles, with stand-ins for the compilers and for torch:
C and C++ callers need no torch, and the tensors' module follows the torch that is
installed."""
import importlib.util
import os
import stat
import subprocess
import types

import pytest

from sequence_re_layout_gb300 import build

COMPILER = """#!/bin/sh
# writes its own name to the file after -o, unless told to fail
[ -e "$0.fails" ] && exit 3
while [ $# -gt 1 ]; do
  [ "$1" = -o ] && echo "$0" > "$2"
  shift
done
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Paths of a package of its own, compilers that only leave a file, and a torch."""
    t = types.SimpleNamespace(root=tmp_path, torch=tmp_path / "torch")
    for name in ("nvcc", "g++"):
        exe = tmp_path / "bin" / name
        exe.parent.mkdir(exist_ok=True)
        exe.write_text(COMPILER)
        exe.chmod(exe.stat().st_mode | stat.S_IXUSR)
    for name, file in (("LIB_PATH", "libbasp.so"), ("DEBUG_LIB_PATH", "libbasp_debug.so"),
                       ("TORCH_OPS_PATH", "_torch_ops.so"), ("TORCH_VERSION_PATH", "_torch_ops.built_with")):
        monkeypatch.setattr(build, name, str(tmp_path / file), raising=False)
    monkeypatch.setattr(build, "_nvcc", lambda: str(tmp_path / "bin" / "nvcc"))
    monkeypatch.setenv("PATH", str(tmp_path / "bin"), prepend=os.pathsep)
    (t.torch / "lib").mkdir(parents=True)
    (t.torch / "lib" / "libtorch_cuda.so").touch()
    (t.torch / "__init__.py").touch()
    (t.torch / "version.py").write_text("__version__ = '1'\n")
    t.spec = types.SimpleNamespace(origin=str(t.torch / "__init__.py"))
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: t.spec if n == "torch" else find(n, *a))
    return t


def built(t):
    return sorted(p.name for p in t.root.iterdir() if p.is_file())


def test_everything(tree):
    assert build.build_library() == build.LIB_PATH
    assert built(tree) == ["_torch_ops.built_with", "_torch_ops.so", "libbasp.so", "libbasp_debug.so"]


def test_without_torch(tree):
    """libbasp.so needs nvcc alone."""
    tree.spec = None
    (tree.root / "bin" / "g++").unlink()
    assert build.build_library() == build.LIB_PATH
    assert built(tree) == ["libbasp.so", "libbasp_debug.so"]


def test_torch_without_cuda(tree):
    (tree.torch / "lib" / "libtorch_cuda.so").unlink()
    build.build_library()
    assert built(tree) == ["libbasp.so", "libbasp_debug.so"]


def test_nothing_to_do_and_another_torch(tree, monkeypatch):
    build.build_library()
    started = []
    popen = subprocess.Popen
    monkeypatch.setattr(subprocess, "Popen", lambda c, *a, **k: (started.append(c[0]), popen(c, *a, **k))[1])
    build.build_library()
    assert started == []
    (tree.torch / "version.py").write_text("__version__ = '2'\n")
    build.build_library()
    assert started == ["g++"]
    build.build_library()
    assert started == ["g++"]


@pytest.mark.parametrize("missing", [False, True])
def test_a_module_that_does_not_compile_leaves_the_libraries(tree, missing, monkeypatch):
    if missing:
        monkeypatch.setattr(build, "_torch_command", lambda out, torch: [str(tree.root / "no-such-compiler")])
    else:
        (tree.root / "bin" / "g++.fails").touch()
    with pytest.raises((subprocess.CalledProcessError, OSError)):
        build.build_library()
    assert built(tree) == ["libbasp.so", "libbasp_debug.so"]
