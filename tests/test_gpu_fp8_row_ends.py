"""What the 8-bit product writes of C ends where C ends: every remainder of its
columns, rows that TMA can address and rows that it cannot, next to memory that
must stay as it is; the values against 64 bits (tolerances: tests/test_gpu_fp8.py)."""
import pytest
import torch

import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import fp8
from test_gpu_fp8 import _built, check_product, f64, quantized, random          # noqa: F401

pytestmark = pytest.mark.gpu


def check_in_store(a, a64, b, b64, K, out, pad, bias):
    """The product into the first columns and rows of a larger store."""
    M, N = a64.shape[0], b64.shape[0]
    store = torch.full((M + 2, N + pad), 7.0, dtype=out, device="cuda")
    c = store[:M, :N]
    assert fp8.matmul(a, b, bias=bias, out=c) is c
    assert bool((store[:, N:] == 7).all()) and bool((store[M:] == 7).all())
    check_product(c, a64, b64, K, None if bias is None else f64(bias))


# tiles 16, 32, 32, 64 and 128 wide, and pairs
@pytest.mark.parametrize("M,N,K", [(17, 256, 64), (60, 6400, 200), (1000, 1536, 200), (101, 19968, 300),
                                   (700, 6016, 300), (1021, 2976, 1543)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_every_remainder_of_a_row(M, N, K, out):
    a, a64 = quantized(M, K, 1, 1)
    a64 = a64 * 2.0 ** -20                                     # fp16 ends at 65504
    a.scales.view(torch.uint8).sub_(20)
    b, b64 = quantized(N + 33, K, 1, 2)
    for n in [N + r for r in (list(range(34)) if M < 100 else [1, 2, 7, 8, 9, 15, 20, 24, 31])]:
        bn = fp8.Quantized(b.data[:n], b.scales[:n])
        bias = random(1, n, out, n, 0.5)[0] if n % 2 else None
        # rows at multiples of 16 bytes, and not
        check_in_store(a, a64, bn, b64[:n], K, out, -n % 8 + 8, bias)
        check_in_store(a, a64, bn, b64[:n], K, out, -n % 8 + 9, bias)


@pytest.mark.parametrize("N", [1, 5, 7, 8, 9, 23])
def test_few_columns(N):
    a, a64 = quantized(300, 200, 1, 1)
    b, b64 = quantized(N, 200, 1, 2)
    check_in_store(a, a64, b, b64, 200, torch.bfloat16, -N % 8 + 8, None)


@pytest.mark.parametrize("N", [131072, 131073, 131079, 131084])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16])
def test_one_row(N, out):
    """A single row's stride is free; the row still ends after N."""
    a, a64 = quantized(1, 256, 1, 1)
    a64 = a64 * 2.0 ** -20
    a.scales.view(torch.uint8).sub_(20)
    b, b64 = quantized(N, 256, 128, 2)
    store = torch.full((N + 16,), 7.0, dtype=out, device="cuda")
    c = store[:N].view(1, N)
    fp8.matmul(a, b, out=c)
    assert bool((store[N:] == 7).all())
    check_product(c, a64, b64, 256)


def poisoned(q):
    """The same matrix in storage whose every other byte is NaN, scales too."""
    rows, cols = q.shape
    srows, blocks = q.scales.shape
    d = torch.full((rows + 1, -(-cols // 16) * 16 + 16), 0x7f, dtype=torch.uint8, device="cuda")
    s = torch.full((srows + 1, -(-blocks // 4) * 4 + 4), 0xff, dtype=torch.uint8, device="cuda")
    d[:rows, :cols], s[:srows, :blocks] = q.data.view(torch.uint8), q.scales.view(torch.uint8)
    return fp8.Quantized(d.view(torch.float8_e4m3fn)[:rows, :cols], s.view(torch.float8_e8m0fnu)[:srows, :blocks],
                         q.block_rows)


# few tokens, a tile alone, shared K, pairs
@pytest.mark.parametrize("M,N,K", [(3, 50, 128), (17, 257, 128), (20, 100, 2560), (1021, 2999, 1536)])
def test_bytes_past_a_row_are_not_used(M, N, K):
    for k in [K + r for r in (list(range(1, 34)) + [64, 127] if M < 100 else [1, 2, 3, 7, 15, 20])]:
        a, a64 = quantized(M, k, 1, 1)
        b, b64 = quantized(N, k, 128, 2)
        c = fp8.matmul(poisoned(a), poisoned(b), out_dtype=torch.float32)
        check_product(c, a64, b64, k)


def test_zz_no_wait_ran_out():
    assert basp.basp_matmul_fp8_timeouts() == 0
