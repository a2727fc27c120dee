"""The 8-bit product on every path of its kernel (tests/product_shapes.py), against
64 bits: widths alone and in pairs, accumulators used again, segments of a long
sum, K shared by CTAs, results by TMA and one by one.

The plain form is a product in 64 bits of the values that the operands stand for.
Tolerances as in tests/test_gpu_fp8.py: u(t) = finfo(t).eps / 2 for the last
rounding; before it at most one rounding or truncation, 2^-23, for each 32 terms of
the sum over K, each part and each term added to it, of at most the sum of magnitudes;
2^-25 is the last step of fp16."""
import functools

import pytest
import torch

import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import fp8
from product_shapes import PATHS
from test_gpu_fp8 import _built                             # noqa: F401

pytestmark = pytest.mark.gpu


def matrix(rows, cols, block_rows, seed, shift):
    """An 8-bit matrix with exponents of its own, and its 64-bit values."""
    g = torch.Generator().manual_seed(seed)
    data = (torch.randn(rows, cols, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    exps = torch.randint(-9, 10, (-(-rows // block_rows), -(-cols // 128)), generator=g) - shift
    q = fp8.Quantized.empty(rows, cols, block_rows)
    q.data.view(torch.uint8).copy_(data.view(torch.uint8))
    q.scales.view(torch.uint8).copy_((exps + 127).to(torch.uint8))
    spread = torch.exp2(exps.double()).repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q, data.double().cuda() * spread.cuda()


@functools.lru_cache(maxsize=1)
def operands(M, N, K):
    """a, b, their product and its sum of magnitudes; in all 2^-28, so that every
    result is in fp16's range."""
    a, a64 = matrix(M, K, 1, 1, 16)
    b, b64 = matrix(N, K, 1 if K // 2 % 2 else 128, 2, 12)
    return a, b, a64 @ b64.T, a64.abs() @ b64.abs().T


def check(c, want, size, K):
    tol = torch.finfo(c.dtype).eps / 2 * want.abs() + (-(-K // 32) + 16) * 2.0 ** -23 * size + 2.0 ** -25
    off = (c.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("shape", PATHS, ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
def test_product(shape, out):
    M, N, K = shape
    a, b, want, size = operands(*shape)
    g = torch.Generator().manual_seed(3)
    bias, base = torch.randn(N, generator=g).to(out).cuda(), torch.randn(M, N, generator=g).to(out).cuda()
    # rows back to back
    first = fp8.matmul(a, b, out_dtype=out)
    check(first, want, size, K)
    assert torch.equal(fp8.matmul(a, b, out_dtype=out), first)
    # rows that TMA can address, with a bias
    store = torch.full((M, -(-N // 8) * 8 + 8), 7.0, dtype=out, device="cuda")
    c = store[:, :N]
    fp8.matmul(a, b, bias=bias, out=c)
    biased, more = want + bias.double(), size + bias.double().abs()
    check(c, biased, more, K)
    assert bool((store[:, N:] == 7).all())
    # the same added to what is there
    c.copy_(base)
    fp8.matmul(a, b, bias=bias, out=c, accumulate=True)
    check(c, biased + base.double(), more + base.double().abs(), K)
    assert bool((store[:, N:] == 7).all())


def test_zz_no_wait_ran_out():
    assert basp.basp_matmul_fp8_timeouts() == 0
