"""The 8-bit operators as torch code sees them: tensors without elements, and what
autograd is told of a tensor that a call writes to."""
import pytest
import torch

import sequence_re_layout_gb300 as basp                     # noqa: F401
from sequence_re_layout_gb300 import fp8
from test_gpu_fp8 import _built                             # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_no_columns(quantized, dtype):
    """rstd = (0 / 0 + eps)^-1/2, whatever the memory held before."""
    used = torch.full((4096,), 5.0, device="cuda")
    del used
    x, w = torch.empty(4096, 0, dtype=dtype, device="cuda"), torch.empty(0, dtype=dtype, device="cuda")
    y, h, rstd = fp8.rmsnorm(x, w, quantized=quantized)
    assert y.shape == h.shape == (4096, 0) and rstd.shape == (4096,)
    assert bool(torch.isnan(rstd).all())
    y, _, rstd = fp8.rmsnorm(x[:0], w, quantized=quantized)
    assert y.shape == (0, 0) and rstd.shape == (0,)
