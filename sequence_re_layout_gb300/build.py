"""Compile the C-ABI library in-tree with nvcc for sm_103a: ``libbasp.so``
(release) and ``libbasp_debug.so`` (every access of the re-layout kernel
bounds-checked); and ``_torch_ops.so``, the 8-bit operators' calls on torch
tensors (host code only, against the installed torch)."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libbasp.so")
DEBUG_LIB_PATH = os.path.join(PKG, "libbasp_debug.so")
TORCH_OPS_PATH = os.path.join(PKG, "_torch_ops.so")
TORCH_OPS_SOURCE = os.path.join(CSRC, "torch_ops.cpp")
SOURCES = ["layout.cpp", "relayout.cu", "rmsnorm.cu", "quantize.cu", "matmul.cu"]
HEADERS = [os.path.join(INCLUDE, h) for h in ("basp.h", "basp_debug.h", "basp_fp8.h")] + \
    [os.path.join(CSRC, h) for h in ("layout_internal.h", "relayout_kernel.cuh", "scratch_cache.h",
                                     "fp8_common.cuh", "matmul_plan.h", "matvec.cuh", "tcgen05.cuh")]

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-shared",
    "--threads", "8",       # the sources side by side
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _stale(path, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def _command(out, extra, verbose):
    cmd = [_nvcc()] + NVCC_FLAGS + extra + ["-I", INCLUDE, "-o", out] + \
        [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def _torch_command(out):
    # found without importing torch, which takes longer than the compilation
    import importlib.util
    import sysconfig
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    libs = os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
            "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda or "/usr/local/cuda", "include"),
            TORCH_OPS_SOURCE, "-o", out, "-L", libs, "-Wl,-rpath," + libs,
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build ``libbasp.so``, ``libbasp_debug.so`` and ``_torch_ops.so`` next to
    this file (side by side) if missing or out of date; return the release
    library's path."""
    jobs = []
    sources = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    for path, deps, command in (
            (LIB_PATH, sources, lambda tmp: _command(tmp, [], verbose)),
            (DEBUG_LIB_PATH, sources, lambda tmp: _command(tmp, ["-DBASP_CHECK_BOUNDS=1"], verbose)),
            (TORCH_OPS_PATH, [TORCH_OPS_SOURCE] + HEADERS[:3], _torch_command)):
        if force or _stale(path, deps):
            tmp = path + ".tmp%d" % os.getpid()
            jobs.append((subprocess.Popen(command(tmp)), tmp, path))
    failed = None
    for proc, tmp, path in jobs:
        if proc.wait() != 0:
            failed = proc
        elif failed is None:
            os.replace(tmp, path)
    if failed is not None:
        raise subprocess.CalledProcessError(failed.returncode, failed.args[0])
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
