"""Compile the C-ABI library in-tree with nvcc for sm_103a: ``libbasp.so``
(release) and ``libbasp_debug.so`` (every access of the re-layout kernel
bounds-checked).  They need nvcc alone.  Where torch is installed, also
``_torch_ops.so``, the 8-bit operators' calls on torch tensors (host code only,
against that torch)."""
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
TORCH_VERSION_PATH = os.path.join(PKG, "_torch_ops.built_with")
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


def _torch_dir():
    """The installed torch with CUDA, or None.  Found without importing it, which
    takes longer than the compilation."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    torch = os.path.dirname(spec.origin)
    return torch if os.path.exists(os.path.join(torch, "lib", "libtorch_cuda.so")) else None


def _torch_version(torch) -> str:
    """What _torch_ops.so was built against: it uses torch's C++ interface, which
    changes from one version to the next."""
    with open(os.path.join(torch, "version.py")) as f:
        return torch + "\n" + f.read()


def _torch_is_other(torch) -> bool:
    try:
        with open(TORCH_VERSION_PATH) as f:
            return f.read() != _torch_version(torch)
    except OSError:
        return True


def _torch_command(out, torch):
    import sysconfig
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    libs = os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
            "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda or "/usr/local/cuda", "include"),
            TORCH_OPS_SOURCE, "-o", out, "-L", libs, "-Wl,-rpath," + libs,
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Build ``libbasp.so``, ``libbasp_debug.so`` and, where torch is installed,
    ``_torch_ops.so`` next to this file (side by side) if missing or out of date;
    return the release library's path.  What compiles is put in place also where
    something else does not; that is an error afterwards."""
    sources = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    commands = []
    for path, extra in ((LIB_PATH, []), (DEBUG_LIB_PATH, ["-DBASP_CHECK_BOUNDS=1"])):
        if force or _stale(path, sources):
            commands.append((path, _command(path + ".tmp%d" % os.getpid(), extra, verbose)))
    torch = _torch_dir()
    if torch is not None and (force or _stale(TORCH_OPS_PATH, [TORCH_OPS_SOURCE] + HEADERS[:3]) or
                              _torch_is_other(torch)):
        commands.append((TORCH_OPS_PATH, _torch_command(TORCH_OPS_PATH + ".tmp%d" % os.getpid(), torch)))
    jobs, failed = [], None
    for path, command in commands:
        try:
            jobs.append((path, command, subprocess.Popen(command)))
        except OSError as e:                    # no such compiler
            failed = e
    for path, command, proc in jobs:
        if proc.wait() != 0:
            failed = subprocess.CalledProcessError(proc.returncode, command[0])
            continue
        os.replace(path + ".tmp%d" % os.getpid(), path)
        if path == TORCH_OPS_PATH:
            with open(TORCH_VERSION_PATH, "w") as f:
                f.write(_torch_version(torch))
    if failed is not None:
        raise failed
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
