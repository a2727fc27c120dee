"""The product's host-checkable parts (csrc/matmul_plan.h), by a C++ program
(tests/c/matmul_plan_test.cpp); no GPU."""
import os
import subprocess

import pytest

from product_shapes import PATHS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("c") / "matmul_plan_test")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-o", exe,
                    os.path.join(ROOT, "tests", "c", "matmul_plan_test.cpp"),
                    "-I", os.path.join(ROOT, "sequence_re_layout_gb300", "csrc"),
                    "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(CUDA, "include")], check=True)
    return exe


def run(*command):
    r = subprocess.run(command, capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_no_buffer_is_written_while_a_store_reads_it(program):
    assert "matmul_plan ok" in run(program)


def test_compared_products_take_every_path(program):
    """The products that tests/test_gpu_fp8_paths.py compares with 64 bits are on
    the paths that they are there for, on 152 SMs, and leave none out."""
    lines = run(program, "152", *(str(n) for shape in PATHS for n in shape)).splitlines()
    got = {shape: tuple(int(n) for n in line.split()) for shape, line in zip(PATHS, lines)}
    assert got == PATHS
    plans = list(PATHS.values())
    # every width, alone and in pairs; every split of K
    assert {(p[0], p[1]) for p in plans} == {(16, 0), (32, 0), (64, 0), (128, 0), (192, 1), (224, 1)}
    assert {p[2] for p in plans} == {1, 2, 4}
    for pair in (0, 1):
        # accumulators reused, and reused again; 32-bit results of several
        # segments of 16 blocks of K, in more than one tile of a CTA
        assert any(p[1] == pair and p[3] >= 5 for p in plans)
        assert any(p[1] == pair and p[2] == 1 and p[4] > 32 for p in plans)
    assert any(p[2] == 1 and p[3] >= 2 and p[4] > 32 for p in plans)
    assert any(p[2] > 1 and p[4] > 16 for p in plans)
