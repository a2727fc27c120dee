"""How the norm rounds: y = (h * rstd) * weight, each product rounded to 32 bits, in
every one of its kernels, so that a row's values do not depend on how many rows
there are beyond the order in which its sum is taken (which rstd shows).  Bit for
bit against the same two products by torch, from the rstd that the call returned."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
from sequence_re_layout_gb300 import fp8
from test_gpu_fp8 import _built, f64, random, values_and_exps            # noqa: F401

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def check(x, w, residual=None):
    y, h, rstd = fp8.rmsnorm(x, w, residual=residual, eps=1e-5, quantized=False)
    q, h2, rstd2 = fp8.rmsnorm(x, w, residual=residual, eps=1e-5)
    assert torch.equal(rstd, rstd2) and torch.equal(h, h2)
    y32 = h.float() * rstd[:, None] * w.float()
    assert torch.equal(y, y32.to(x.dtype))
    v, e = values_and_exps(q)
    rv, re = ref.quantize(f64(y32), 1)
    assert np.array_equal(e, re) and np.array_equal(v, rv)


# few rows and many; 16 bytes a load with 1, 2 and 4 of them a thread, elements one
# at a time, rows too long for registers
@pytest.mark.parametrize("rows,cols", [(3, 2048), (400, 2048), (400, 40), (400, 1000), (310, 5120), (310, 9000),
                                       (5, 9000), (700, 129), (310, 4099), (305, 16392)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("more", [False, True])
def test_two_products(rows, cols, dtype, more):
    x, r = random(rows, cols, dtype, 1, 1.0), random(rows, cols, dtype, 2, 1.0) if more else None
    check(x, random(1, cols, torch.float32 if more else dtype, 3, 0.5)[0], r)


@pytest.mark.parametrize("rows", [3, 400])
def test_weights_far_from_one(rows):
    """h * weight would leave the range of 32 bits, h * rstd * weight does not."""
    x = random(rows, 512, torch.float32, 1, 1.0)
    for scale, weight in ((2.0 ** 60, 2.0 ** 90), (2.0 ** 50, 2.0 ** 90), (2.0 ** -50, 2.0 ** -90)):
        w = torch.full((512,), weight, device="cuda")
        check(x * scale, w)
        y, _, rstd = fp8.rmsnorm(x * scale, w, eps=0.0, quantized=False)
        if scale == 2.0 ** 60:                     # 512 squares of 2^120 are past 2^128: the root of their sum is zero
            assert bool((rstd == 0).all()) and bool((y == 0).all())
        else:
            assert bool(torch.isfinite(y).all()) and bool((y != 0).all())
