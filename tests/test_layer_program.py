"""A C++ program (tests/c/layer_example.cpp) built with g++ against include/basp.hpp
and libbasp.so: layer norm, attention and AdamW as a C++ caller uses them."""
import os
import subprocess

import pytest

from sequence_re_layout_gb300.build import LIB_PATH, build_library
from test_fp8_program import CUDA, ROOT, run


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    build_library()
    exe = str(tmp_path_factory.mktemp("c") / "layer_example")
    libdir, cudart = os.path.dirname(LIB_PATH), os.path.join(CUDA, "lib64")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-o", exe,
                    os.path.join(ROOT, "tests", "c", "layer_example.cpp"), "-I", os.path.join(ROOT, "include"),
                    "-isystem", os.path.join(CUDA, "include"), "-L", libdir, "-lbasp", "-L", cudart, "-lcudart",
                    "-Wl,-rpath," + libdir, "-Wl,-rpath," + cudart], check=True)
    return exe


def test_host_checks(program):
    assert "layer_example ok" in run(program)


@pytest.mark.gpu
def test_on_gpu(program):
    assert "layer_example ok" in run(program, "gpu")
