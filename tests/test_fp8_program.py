"""A C++ program (tests/c/fp8_example.cpp) built with g++ against
include/basp.hpp and libbasp.so: the 8-bit projections as a C++ caller uses
them.  And, without a GPU, what the differentiable forms and the example refuse."""
import os
import subprocess
import sys

import pytest
import torch

from sequence_re_layout_gb300 import autograd, fp8
from sequence_re_layout_gb300.build import LIB_PATH, build_library

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    build_library()
    exe = str(tmp_path_factory.mktemp("c") / "fp8_example")
    libdir, cudart = os.path.dirname(LIB_PATH), os.path.join(CUDA, "lib64")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-o", exe,
                    os.path.join(ROOT, "tests", "c", "fp8_example.cpp"), "-I", os.path.join(ROOT, "include"),
                    "-isystem", os.path.join(CUDA, "include"), "-L", libdir, "-lbasp", "-L", cudart, "-lcudart",
                    "-Wl,-rpath," + libdir, "-Wl,-rpath," + cudart], check=True)
    return exe


def run(*command):
    r = subprocess.run(command, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_host_checks(program):
    assert "fp8_example ok" in run(program)


@pytest.mark.gpu
def test_on_gpu(program):
    assert "fp8_example ok" in run(program, "gpu")


def test_an_8_bit_weight_has_no_gradient():
    w = fp8.Quantized.empty(8, 128, 128, device="cpu")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="no gradient"):
        autograd.linear_fp8(x, w)
    with pytest.raises(TypeError, match="no gradient"):
        autograd.rmsnorm_linear_fp8(x, torch.ones(128, dtype=torch.bfloat16), w)


def test_example_has_help():
    assert "--workload" in run(sys.executable, os.path.join(ROOT, "examples", "attention_layer.py"), "--help")
