"""Matrices of more than 2^31 elements: the last rows get what they get alone.  The
same kernels run on the parts (many rows, whole tiles), and a row's or a tile's
results depend on nothing else, so they agree bit for bit; the product's parts have
other tiles, whose 16-bit results are each within a rounding and a 32-bit sum of 64 bits."""
import pytest
import torch

from sequence_re_layout_gb300 import fp8
from test_gpu_fp8 import _built                             # noqa: F401

pytestmark = pytest.mark.gpu

ROWS, COLS, LAST = 65536 + 640, 32768, 640                  # 2.2e9 values; whole tiles of 128


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.fixture(scope="module")
def x():
    torch.manual_seed(1)
    x = torch.empty(ROWS, COLS, dtype=torch.bfloat16, device="cuda")
    for part in x.split(4096):
        part.normal_()
    yield x
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cols", [COLS, 16384, COLS - 1])    # two walks a row; loads ahead; elements one by one
def test_norm(x, cols):
    w = torch.randn(cols, device="cuda").bfloat16()
    part = x[:, COLS - cols:]
    y, h, rstd = fp8.rmsnorm(part, w, residual=part)
    y2, h2, rstd2 = fp8.rmsnorm(part[-LAST:], w, residual=part[-LAST:])
    assert torch.equal(h[-LAST:], h2) and torch.equal(rstd[-LAST:], rstd2)
    assert same(y.data[-LAST:], y2.data) and same(y.scales[-LAST:], y2.scales)
    del y
    dx, dw = fp8.rmsnorm_backward(part, h, rstd, w)
    assert torch.equal(dx[-LAST:], fp8.rmsnorm_backward(part[-LAST:], h2, rstd2, w)[0])
    assert bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("cols", [COLS, COLS - 1])
def test_quantize(x, block_rows, cols):
    part = x[:, :cols]
    q, qt = fp8.quantize(part, block_rows=block_rows, transposed=True)
    q2, qt2 = fp8.quantize(part[-LAST:], block_rows=block_rows, transposed=True)
    n = LAST // block_rows
    assert same(q.data[-LAST:], q2.data) and same(q.scales[-n:], q2.scales)
    assert same(qt.data[:, -LAST:], qt2.data) and same(qt.scales[:, -LAST // 128:], qt2.scales)
    if block_rows == 1:
        assert same(fp8.quantize(part).data[-LAST:], q2.data)


@pytest.mark.parametrize("out,cols", [(torch.bfloat16, COLS), (torch.bfloat16, COLS - 1), (torch.float32, COLS)])
def test_product(x, out, cols):
    a, b = fp8.quantize(x[:, :200]), fp8.quantize(x[:cols, 256:456], block_rows=128)
    c = fp8.matmul(a, b, out_dtype=out)[-LAST:]
    a64, b64 = a.dequantize()[-LAST:].double(), b.dequantize().double()
    want, size = a64 @ b64.T, a64.abs() @ b64.abs().T
    tol = torch.finfo(out).eps / 2 * want.abs() + (200 // 32 + 17) * 2.0 ** -23 * size
    assert bool(((c.double() - want).abs() <= tol).all())


def test_operand(x):
    """An operand of more than 2^31 values."""
    b = fp8.quantize(x)
    a = fp8.quantize(x[:20])
    c = fp8.matmul(a, b, out_dtype=torch.float32)[:, -LAST:]
    a64 = a.dequantize().double()
    b64 = (b.data[-LAST:].double().view(LAST, -1, 128) * b.scales[-LAST:].double()[:, :, None]).view(LAST, COLS)
    want, size = a64 @ b64.T, a64.abs() @ b64.abs().T
    assert bool(((c.double() - want).abs() <= (COLS // 32 + 16) * 2.0 ** -23 * size + 2.0 ** -24 * want.abs()).all())
