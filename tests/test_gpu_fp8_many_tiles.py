"""The 8-bit product where a CTA works through several tiles one after the
other, against 64 bits: results on their way out of one tile meet the next.

Tolerances as in tests/test_gpu_fp8.py: u(t) = finfo(t).eps / 2 for the last
rounding; before it at most one rounding or truncation, 2^-23, for each 32 terms of
the sum over K, of at most the sum of magnitudes."""
import pytest
import torch

import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import fp8
from test_gpu_fp8 import _built, check_product, quantized          # noqa: F401

pytestmark = pytest.mark.gpu

REPEATS = 20


@pytest.mark.parametrize("M,N,K", [
    # tiles of 32 tokens, two to five a CTA; short sums, so that one tile's
    # results go out right after the other's
    (32, 40000, 128), (287, 4096, 1024), (1195, 2432, 128), (201, 5120, 1024),
    # tiles of 16, two to seven a CTA: an output vocabulary, a short prompt
    (96, 8192, 128), (16, 32000, 300), (8, 131072, 256), (9, 50008, 64)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_results_of_consecutive_tiles(M, N, K, out):
    a, a64 = quantized(M, K, 1, 1)
    b, b64 = quantized(N, K, 128, 2)
    if out == torch.float16:                                   # fp16 ends at 65504
        a64, b64 = a64 * 2.0 ** -12, b64 * 2.0 ** -8
        a.scales.view(torch.uint8).sub_(12)
        b.scales.view(torch.uint8).sub_(8)
    first = fp8.matmul(a, b, out_dtype=out)
    check_product(first, a64, b64, K)
    for _ in range(REPEATS):
        assert torch.equal(fp8.matmul(a, b, out_dtype=out), first)


def test_zz_no_wait_ran_out():
    assert basp.basp_matmul_fp8_timeouts() == 0
