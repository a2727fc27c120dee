"""The product's host-checkable parts (csrc/matmul_plan.h), by a C++ program
(tests/c/matmul_plan_test.cpp); no GPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("c") / "matmul_plan_test")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-o", exe,
                    os.path.join(ROOT, "tests", "c", "matmul_plan_test.cpp"),
                    "-I", os.path.join(ROOT, "sequence_re_layout_gb300", "csrc")], check=True)
    return exe


def test_no_buffer_is_written_while_a_store_reads_it(program):
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert "matmul_plan ok" in r.stdout
