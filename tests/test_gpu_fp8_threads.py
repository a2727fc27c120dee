"""Several host threads in the norm's calls at once (tests/c/fp8_threads.cpp): what
one thread's launch needs of a kernel is not taken back by another's."""
import os
import subprocess

import pytest

from sequence_re_layout_gb300.build import LIB_PATH, build_library

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_norms_of_different_length_side_by_side(tmp_path):
    build_library()
    exe, libdir, cudart = str(tmp_path / "fp8_threads"), os.path.dirname(LIB_PATH), os.path.join(CUDA, "lib64")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-pthread", "-o", exe,
                    os.path.join(ROOT, "tests", "c", "fp8_threads.cpp"), "-I", os.path.join(ROOT, "include"),
                    "-isystem", os.path.join(CUDA, "include"), "-L", libdir, "-lbasp", "-L", cudart, "-lcudart",
                    "-Wl,-rpath," + libdir, "-Wl,-rpath," + cudart], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert "fp8_threads ok" in r.stdout
