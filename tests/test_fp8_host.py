"""CPU checks of the 8-bit operators' C ABI (include/basp_fp8.h): exported
symbols, and refusals, which all happen before anything reaches a GPU."""
import os
import re

import pytest
import torch

import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import fp8
from sequence_re_layout_gb300.build import build_library

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "include", "basp_fp8.h")
BF16, FP32, FP16, FP8 = (basp.DTYPE_CODES[n] for n in ("bf16", "fp32", "fp16", "fp8"))
OK = 0
INVALID, ALIGN, ALIAS, WORKSPACE, LARGE = (
    basp.BASP_ERR_INVALID_ARG, basp.BASP_ERR_ALIGNMENT, basp.BASP_ERR_ALIASING,
    basp.BASP_ERR_WORKSPACE, basp.BASP_ERR_TOO_LARGE)
GiB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return basp.load_library()


def at(n):
    """An address that no call here dereferences: everything it is given to is
    refused, or has nothing to do."""
    return (1 << 40) + n * GiB


def q8(n, rows, cols, block_rows=1, **change):
    blocks = -(-cols // 128)
    f = dict(data=at(n), scales=at(n) + GiB // 2, rows=rows, cols=cols, pitch=-(-cols // 16) * 16,
             scale_pitch=-(-blocks // 4) * 4, block_rows=block_rows)
    f.update(change)
    return basp.basp_fp8_matrix(**f)


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(basp_\w+)\s*\(", text))
    assert names == set(basp.FP8_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


NORM = dict(dtype=BF16, rows=4, cols=256, x=at(1), xs=256, r=at(2), rs=256, w=at(3), wd=BF16, eps=1e-6,
            h=at(4), hs=256, y=at(5), ys=256, q=None, rstd=at(6), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), OK), (dict(cols=0, q=q8(7, 4, 0)), OK),
    (dict(rows=0, x=None, r=None, h=None, y=at(5), rstd=None), OK),
    (dict(dtype=FP8), INVALID), (dict(dtype=9), INVALID), (dict(wd=FP16), INVALID), (dict(wd=FP8), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=-1), INVALID), (dict(rows=1 << 31), LARGE), (dict(cols=1 << 31), LARGE),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None, q=None), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xs=255), INVALID), (dict(hs=-256), INVALID), (dict(xs=1 << 60), LARGE),
    (dict(x=at(1) + 1), ALIGN), (dict(rstd=at(6) + 2), ALIGN),
    (dict(y=at(1)), ALIAS), (dict(y=at(4) + 512), ALIAS), (dict(h=at(1) + 512), ALIAS),
    (dict(h=at(1), hs=512), ALIAS), (dict(h=at(3)), ALIAS), (dict(rstd=at(3)), ALIAS),
    (dict(q=q8(7, 4, 128)), INVALID), (dict(q=q8(7, 3, 256)), INVALID),
    (dict(q=q8(7, 4, 256, 128)), INVALID), (dict(q=q8(7, 4, 256, 2)), INVALID),
    (dict(q=q8(7, 4, 256, data=None)), INVALID), (dict(q=q8(7, 4, 256, scales=None)), INVALID),
    (dict(q=q8(7, 4, 256, pitch=240)), INVALID), (dict(q=q8(7, 4, 256, pitch=264)), ALIGN),
    (dict(q=q8(7, 4, 256, scale_pitch=1)), INVALID), (dict(q=q8(7, 4, 256, scale_pitch=6)), ALIGN),
    (dict(q=q8(7, 4, 256, data=at(7) + 8)), ALIGN), (dict(q=q8(7, 4, 256, scales=at(8) + 2)), ALIGN),
    (dict(q=q8(7, 4, 256, data=at(5))), ALIAS), (dict(q=q8(7, 4, 256, scales=at(7) + 512)), ALIAS),
])
def test_rmsnorm_refusals(lib, change, status):
    a = dict(NORM)
    a.update(change)
    assert lib.basp_rmsnorm(*a.values()) == status


BACK = dict(dtype=BF16, rows=4, cols=256, dy=at(1), dys=256, h=at(2), hs=256, rstd=at(3), w=at(4), wd=FP32,
            dh=at(5), dhs=256, dx=at(6), dxs=256, dw=at(7), ws=at(8), wsb=4 * 256 * 4, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(cols=0), OK), (dict(rows=0, dw=None), OK),
    (dict(dtype=FP8), INVALID), (dict(wd=BF16 + 7), INVALID), (dict(rows=1 << 31), LARGE),
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), INVALID),
    (dict(dx=None), INVALID), (dict(dxs=100), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=4 * 256 * 4 - 1), WORKSPACE), (dict(ws=at(8) + 4), ALIGN),
    (dict(dx=at(2)), ALIAS), (dict(dx=at(1) + 512), ALIAS), (dict(dw=at(4)), ALIAS), (dict(ws=at(1)), ALIAS),
    (dict(dx=at(5), dxs=512), ALIAS), (dict(dw=at(8)), ALIAS), (dict(dw=at(7) + 2), ALIGN),
])
def test_rmsnorm_backward_refusals(lib, change, status):
    a = dict(BACK)
    a.update(change)
    assert lib.basp_rmsnorm_backward(*a.values()) == status


def test_backward_workspace(lib):
    assert basp.basp_rmsnorm_backward_workspace(0, 256) == 0
    assert basp.basp_rmsnorm_backward_workspace(4, 256) == 4 * 256 * 4
    big = basp.basp_rmsnorm_backward_workspace(1 << 20, 256)
    assert big == basp.basp_rmsnorm_backward_workspace(1 << 21, 256)


QUANT = dict(dtype=FP32, rows=130, cols=200, x=at(1), xs=200, q=q8(2, 130, 200), qt=q8(3, 200, 130), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0, q=q8(2, 0, 200), qt=None), OK),
    (dict(q=None, qt=None), INVALID), (dict(dtype=FP8), INVALID), (dict(x=None), INVALID),
    (dict(qt=q8(3, 130, 200)), INVALID), (dict(q=q8(2, 200, 130)), INVALID),
    (dict(qt=q8(3, 200, 130, 128)), INVALID), (dict(xs=199), INVALID), (dict(x=at(1) + 2), ALIGN),
    (dict(cols=-5), INVALID), (dict(rows=1 << 31), LARGE),
    (dict(qt=q8(3, 200, 130, data=at(2))), ALIAS), (dict(q=q8(2, 130, 200, scales=at(1))), ALIAS),
    (dict(q=q8(2, 130, 200, pitch=216)), ALIGN),
])
def test_quantize_refusals(lib, change, status):
    a = dict(QUANT)
    a.update(change)
    assert lib.basp_quantize_fp8(*a.values()) == status


MATMUL = dict(a=q8(1, 33, 200), b=q8(2, 70, 200, 128), bias=at(3), acc=0, dtype=BF16, c=at(4), cs=70, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(a=q8(1, 0, 200)), OK), (dict(b=q8(2, 0, 200)), OK),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(dtype=FP8), INVALID),
    (dict(a=q8(1, 33, 201)), INVALID), (dict(c=None), INVALID), (dict(cs=69), INVALID),
    (dict(a=q8(1, 33, 200, block_rows=64)), INVALID), (dict(b=q8(2, 70, 200, data=None)), INVALID),
    (dict(a=q8(1, 33, 200, data=at(1) + 8)), ALIGN), (dict(a=q8(1, 33, 200, pitch=200)), ALIGN),
    (dict(b=q8(2, 70, 200, scale_pitch=2)), ALIGN), (dict(c=at(4) + 1), ALIGN), (dict(bias=at(3) + 1), ALIGN),
    (dict(a=q8(1, 1 << 31, 200)), LARGE), (dict(c=at(1)), ALIAS), (dict(c=at(3)), ALIAS),
    (dict(c=at(2) + GiB // 2), ALIAS),
])
def test_matmul_refusals(lib, change, status):
    a = dict(MATMUL)
    a.update(change)
    assert lib.basp_matmul_fp8(*a.values()) == status


def test_status_pointer(lib):
    assert lib.basp_matmul_fp8_timeouts(None) == INVALID


def test_python_refusals():
    """What the tensors' calls refuse before they look for a GPU."""
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
    q = fp8.Quantized(torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.ones(4, 1).to(torch.float8_e8m0fnu))
    for call in (lambda: fp8.rmsnorm(x, w), lambda: fp8.rmsnorm(x.double(), w), lambda: fp8.rmsnorm(x, None),
                 lambda: fp8.rmsnorm_backward(x, x, torch.ones(4), w), lambda: fp8.quantize(x),
                 lambda: fp8.quantize(x, block_rows=64), lambda: fp8.quantize(x, rows=False),
                 lambda: fp8.quantize(torch.zeros(())), lambda: fp8.matmul(q, q),
                 lambda: fp8.Quantized.empty(4, 16, 2, "cpu")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        basp.binding.fp8_dtype_code(torch.float64)


def test_torch_module_calls_the_loaded_library(lib):
    import ctypes
    want = [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in basp.FP8_EXPORTS[:5]]
    assert list(basp.binding.fp8_entry_points()) == want
