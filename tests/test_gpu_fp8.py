"""The 8-bit operators on the GPU against their plain 64-bit forms
(tests/fp8_reference.py).

Tolerances.  u(t) = finfo(t).eps / 2 is one rounding to t.  Everything before
the last rounding is in 32 bits: a row's sum of n squares is off by at most
n * 2^-24 of itself, its root by half of that, so a normed value by
(n / 2 + 8) * 2^-24 of itself before it is rounded.  An e4m3 value is off by
half a step: 2^-4 of a normal value, 2^-10 of the scale below.  A product's sum
over K has at most one rounding or truncation, 2^-23, for each 32 terms and
each part of a split, of at most the sum of magnitudes."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import fp8

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sequence_re_layout_gb300.build import build_library
    build_library()


def u(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().float().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def values_and_exps(q):
    """A Quantized as the plain form has it."""
    return f64(q.data), q.scales.cpu().view(torch.uint8).numpy().astype(np.int64) - 127


def random(rows, cols, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(1, cols, generator=g))
    return x.to(dtype).cuda()


def strided(x, pad):
    """The same matrix with `pad` more elements in each row of its storage."""
    big = torch.full((x.shape[0], x.shape[1] + pad), float("nan"), dtype=x.dtype, device=x.device)
    big[:, :x.shape[1]] = x
    return big[:, :x.shape[1]]


SHAPES = [(1, 1), (1, 64), (1, 2048), (3, 127), (2, 128), (5, 129), (33, 260), (700, 256), (401, 1000), (9, 4099),
          (2, 16385), (400, 2048), (310, 5120),
          # many rows that start anywhere: from one column to the longest that stay in registers, and past it
          (1201, 1), (700, 7), (333, 129), (320, 130), (1300, 257), (309, 4099), (310, 9001), (305, 16001),
          (306, 16389), (320, 20000)]


# ---- quantisation -------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (2, 128), (127, 129), (128, 128), (130, 257), (300, 1000),
                                       (1, 4096), (517, 36)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(rows, cols, dtype, block_rows):
    """Bit for bit: the input is exact and a power-of-two scale rounds nothing."""
    x = random(rows, cols, DTYPES[dtype], rows * cols)
    q, qt = fp8.quantize(x, block_rows=block_rows, transposed=True)
    for got, want in ((q, f64(x)), (qt, f64(x).T)):
        v, e = values_and_exps(got)
        rv, re = ref.quantize(want, block_rows)
        assert np.array_equal(e, re)
        assert np.array_equal(v, rv)
    alone, alone_t = fp8.quantize(x, block_rows=block_rows), fp8.quantize(x, block_rows=block_rows, rows=False,
                                                                          transposed=True)
    for a, b in ((alone, q), (alone_t, qt)):
        assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8))
        assert torch.equal(a.scales.view(torch.uint8), b.scales.view(torch.uint8))


@pytest.mark.parametrize("pad", [1, 4, 8])
def test_quantize_strided_input(pad):
    x = random(140, 200, torch.bfloat16, 7)
    want, got = fp8.quantize(x, transposed=True), fp8.quantize(strided(x, pad), transposed=True)
    for a, b in zip(want, got):
        assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8))
        assert torch.equal(a.scales.view(torch.uint8), b.scales.view(torch.uint8))


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extreme_values(block_rows):
    """Zeros, the type's largest and smallest magnitudes, infinities and NaN."""
    x = torch.zeros(130, 384)
    x[0, :128] = torch.finfo(torch.float32).max
    x[1, :128] = -torch.finfo(torch.float32).tiny
    x[2, :128] = 1e-45
    x[129, 5] = float("inf")
    x[129, 6] = float("-inf")
    x[129, 130] = float("nan")
    x[129, 131] = 3.0
    x[4, 256:] = torch.arange(128) * 0.25
    q, qt = fp8.quantize(x.cuda(), block_rows=block_rows, transposed=True)
    for got, want in ((q, f64(x)), (qt, f64(x).T)):
        v, e = values_and_exps(got)
        rv, re = ref.quantize(want, block_rows)
        assert np.array_equal(e, re)
        assert np.array_equal(v, rv, equal_nan=True)


def test_quantize_writes_nothing_past_its_rows():
    x = random(130, 200, torch.bfloat16, 9)
    stores = [torch.full((r, c), 0x55, dtype=torch.uint8, device="cuda")
              for r, c in ((130, 224), (130, 8), (200, 160), (200, 8))]
    q, s, qt, st = stores
    mats = [basp.basp_fp8_matrix(d.data_ptr(), z.data_ptr(), r, c, d.stride(0), 8, 1)
            for d, z, r, c in ((q, s, 130, 200), (qt, st, 200, 130))]
    basp.basp_quantize_fp8(x, mats[0], mats[1], torch.cuda.current_stream())
    torch.cuda.synchronize()
    for store, cols in zip(stores, (200, 2, 130, 2)):
        assert bool((store[:, cols:] == 0x55).all())
    assert np.array_equal(f64(qt.view(torch.float8_e4m3fn)[:, :130]), ref.quantize(f64(x).T, 1)[0])


# ---- norm -----------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(rows, cols, dtype, residual):
    t = DTYPES[dtype]
    x, r = random(rows, cols, t, 1, 1.0), random(rows, cols, t, 2, 1.0) if residual else None
    w = random(1, cols, torch.float32 if rows % 2 else t, 3, 0.5)[0]
    q, h, rstd = fp8.rmsnorm(x, w, residual=r, eps=1e-5)
    y, h2, rstd2 = fp8.rmsnorm(x, w, residual=r, eps=1e-5, quantized=False)
    assert torch.equal(rstd, rstd2) and torch.equal(h, h2)
    want_h = x if r is None else (x.double() + r.double()).float().to(t)     # the sum, rounded to 32 bits and to t
    assert torch.equal(h, want_h)
    ry, rr = ref.norm(f64(h), f64(w), 1e-5)
    slack = (cols / 2 + 8) * F32
    assert (np.abs(f64(rstd) - rr) <= slack * rr).all()
    assert (np.abs(f64(y) - ry) <= (u(t) + slack) * np.abs(ry) + 2.0 ** -25).all()
    v, e = values_and_exps(q)
    rv, re = ref.quantize(ry, 1)
    scale = ref.dequantize(np.ones_like(v), e, 1)
    assert (np.abs(e - re) <= 1).all() and (e != re).mean() < 0.01           # next to a border, either will do
    assert (np.abs(v * scale - ry) <= np.maximum(np.abs(ry) * (2.0 ** -4 + slack), scale * 2.0 ** -10) + 2.0 ** -25).all()


@pytest.mark.parametrize("cols", [200, 201, 2048])
def test_rmsnorm_in_place_and_strided(cols):
    x, r = random(70, cols, torch.bfloat16, 1), random(70, cols, torch.bfloat16, 2)
    w = random(1, cols, torch.bfloat16, 3)[0]
    want, want_h, _ = fp8.rmsnorm(x, w, residual=r)
    for pad in (0, 4, 3):
        xs, rs = strided(x, pad), strided(r, pad)
        got, h, _ = fp8.rmsnorm(xs, w, residual=rs, h=rs)
        assert h is rs and torch.equal(rs, want_h)
        assert torch.equal(got.data.view(torch.uint8), want.data.view(torch.uint8))
    xs = x.clone()
    assert torch.equal(fp8.rmsnorm(xs, w, residual=r, h=xs)[1], want_h) and torch.equal(xs, want_h)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("cols,pad", [(203, 0), (200, 1), (203, 5), (16, 3), (1000, 1), (5, 0), (1, 1)])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_rmsnorm_of_many_rows_that_start_anywhere(cols, pad, dtype, offset):
    """Rows, first elements and strides off the 16-byte grid, all matrices alike
    and then one of them differently, forward and backward, next to memory that
    must stay as it is and must not be used (NaN)."""
    t, rows = DTYPES[dtype], 620
    x, r = random(rows, cols, t, 1, 1.0), random(rows, cols, t, 2, 1.0)
    w = random(1, cols, t, 3, 0.5)[0]
    want, want_h, want_rstd = fp8.rmsnorm(x, w, residual=r)
    want_dx, want_dw = fp8.rmsnorm_backward(x, want_h, want_rstd, w, dh=r)
    rv, re = ref.quantize(ref.norm(f64(want_h), f64(w), 1e-6)[0], 1)

    def placed(m, offset):
        store = torch.full((rows * (cols + pad) + 64,), float("nan"), dtype=t, device="cuda")
        view = store[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        view.copy_(m)
        return store, view

    for other in (offset, offset + 1):                     # alike, or the residual one element further
        (_, xs), (_, rs), (hstore, hs) = placed(x, offset), placed(r, other), placed(r, offset)
        got, h, rstd = fp8.rmsnorm(xs, w, residual=rs, h=hs)
        assert torch.equal(hs, want_h)
        hs.fill_(float("nan"))
        assert bool(torch.isnan(hstore).all())
        v, e = values_and_exps(got)
        assert (e != re).mean() < 0.01 and (v != rv).mean() < 0.01
        # the same bits as the aligned call, but for the order of a row's sum
        assert float((rstd / want_rstd - 1).abs().max()) < 2.0 ** -20
        (_, dys), (_, hs), (_, dhs) = placed(x, offset), placed(want_h, offset), placed(r, other)
        dx, dw = fp8.rmsnorm_backward(dys, hs, want_rstd, w, dh=dhs)
        size = f64(want_rstd)[:, None] * 4 * np.abs(f64(x) * f64(w)).max() + np.abs(f64(r))
        assert (np.abs(f64(dx) - f64(want_dx)) <= 2 * u(t) * np.abs(f64(want_dx)) + (cols + 8) * F32 * size).all()
        scale = (np.abs(f64(x)) * np.abs(f64(want_h)) * f64(want_rstd)[:, None]).sum(0)
        assert (np.abs(f64(dw) - f64(want_dw)) <= 2 * (rows + 8) * F32 * scale + 1e-30).all()


def test_rmsnorm_of_many_ragged_rows_with_infinities():
    """The looked-at values of rows that start anywhere: one infinity makes its
    row's root zero; one NaN its whole row."""
    x = torch.ones(400, 391)
    x[7, 130], x[9, 388], x[11, 0] = float("inf"), float("nan"), float("-inf")
    y, _, _ = fp8.rmsnorm(x.cuda(), torch.ones(391, device="cuda"), quantized=True)
    d = y.dequantize().cpu()
    for row, bad in ((7, 130), (11, 0)):
        assert torch.isnan(d[row, bad]) and int(torch.isnan(d[row]).sum()) == 1
        assert float(d[row].nan_to_num().abs().max()) == 0
    assert bool(torch.isnan(d[9]).all())
    rest = torch.ones(400, dtype=torch.bool)
    rest[[7, 9, 11]] = False
    assert bool((d[rest] == 1).all())
    tiny = torch.full((400, 391), 1e-30, device="cuda")     # 0.03 of the root of eps, times a tiny weight
    y, _, _ = fp8.rmsnorm(tiny, torch.full((391,), 1e-38, device="cuda"), eps=1e-37)
    assert bool(torch.isfinite(y.dequantize()).all())


def test_rmsnorm_leading_dimensions():
    x = random(6, 256, torch.bfloat16, 1).view(2, 3, 256)
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = fp8.rmsnorm(x, w, quantized=False)
    assert y.shape == x.shape and h is x and rstd.shape == (6,)


def test_rmsnorm_rows_of_zeros_infinities_and_nan():
    x = torch.zeros(4, 256)
    x[1, 3], x[2, 200], x[3] = float("inf"), float("nan"), 1.0
    y, _, rstd = fp8.rmsnorm(x.cuda(), torch.ones(256, device="cuda"), eps=1e-6, quantized=True)
    d = y.dequantize().cpu()
    assert bool((d[0] == 0).all())
    assert torch.isnan(d[1, 3]) and bool((d[1, :3] == 0).all())         # inf * 0 and 0 * 0
    assert bool(torch.isnan(d[2]).all()) and bool((d[3] == 1).all())


@pytest.mark.parametrize("rows,cols", SHAPES + [(1300, 384), (3, 8193)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("more", [False, True])
def test_rmsnorm_backward(rows, cols, dtype, more):
    t = DTYPES[dtype]
    h, dy = random(rows, cols, t, 1, 1.0), random(rows, cols, t, 2, 0.5)
    w = random(1, cols, torch.float32 if rows % 2 else t, 3, 0.5)[0]
    dh = random(rows, cols, t, 4, 0.5) if more else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dw = fp8.rmsnorm_backward(dy, h, rstd, w, dh=dh)
    rx, rw = ref.norm_backward(f64(dy), f64(h), f64(rstd), f64(w), None if dh is None else f64(dh))
    # dx is a sum of three terms, one of them with a mean over the row
    g, n = np.abs(f64(dy) * f64(w)), np.abs(f64(h) * f64(rstd)[:, None])
    size = f64(rstd)[:, None] * (g + n * (g * n).mean(1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    assert (np.abs(f64(dx) - rx) <= u(t) * np.abs(rx) + (cols + 8) * F32 * size + 2.0 ** -25).all()
    assert (np.abs(f64(dw) - rw) <= (rows + 8) * F32 * (np.abs(f64(dy)) * n).sum(0) + 1e-30).all()
    again = fp8.rmsnorm_backward(dy, h, rstd, w, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    alone, none = fp8.rmsnorm_backward(dy, h, rstd, w, dh=dh, need_dweight=False)
    assert none is None and torch.equal(alone, dx)


def test_rmsnorm_backward_of_no_rows():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    dx, dw = fp8.rmsnorm_backward(e, e, torch.empty(0, device="cuda"), torch.ones(256, device="cuda"))
    assert dx.shape == (0, 256) and bool((dw == 0).all())


# ---- product ----------------------------------------------------------------------

def quantized(rows, cols, block_rows, seed):
    """An 8-bit matrix with exponents of its own, and its 64-bit values."""
    g = torch.Generator().manual_seed(seed)
    data = (torch.randn(rows, cols, generator=g) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)
    srows, blocks = -(-rows // block_rows), -(-cols // 128)
    exps = torch.randint(-9, 10, (srows, blocks), generator=g)
    q = fp8.Quantized.empty(rows, cols, block_rows)
    q.data.view(torch.uint8).copy_(data.view(torch.uint8))
    q.scales.view(torch.uint8).copy_((exps + 127).to(torch.uint8))
    return q, ref.dequantize(data.double().numpy(), exps.numpy(), block_rows)


def check_product(c, a64, b64, K, bias=None, base=None):
    want, size = a64 @ b64.T, np.abs(a64) @ np.abs(b64).T
    for extra in (bias, base):
        if extra is not None:
            want, size = want + extra, size + np.abs(extra)
    tol = u(c.dtype) * np.abs(want) + (-(-K // 32) + 16) * 2.0 ** -23 * size
    assert (np.abs(f64(c) - want) <= tol + 2.0 ** -25).all(), np.abs((f64(c) - want) / size).max()


@pytest.mark.parametrize("M,N,K", [
    (1, 128, 128), (1, 128, 32), (1, 1, 1), (1, 130, 513), (16, 128, 512), (17, 256, 640), (31, 300, 1000),
    (33, 128, 128), (64, 512, 2048), (65, 129, 127), (127, 257, 129), (128, 128, 4096), (129, 640, 384),
    (255, 1000, 260), (257, 999, 1543), (1000, 77, 128), (2048, 2048, 256), (4099, 1100, 300)])
@pytest.mark.parametrize("out", sorted(DTYPES))
def test_matmul(M, N, K, out):
    a, a64 = quantized(M, K, 1, 1)
    b, b64 = quantized(N, K, 128 if N % 2 else 1, 2)
    scale = 1.0 if out != "fp16" else 2.0 ** -12               # fp16 ends at 65504
    if out == "fp16":
        a64 = a64 * scale
        a.scales.view(torch.uint8).sub_(12)
        b64 = b64 * 2.0 ** -8
        b.scales.view(torch.uint8).sub_(8)
    check_product(fp8.matmul(a, b, out_dtype=DTYPES[out]), a64, b64, K)


@pytest.mark.parametrize("M,N,K", [(1, 300, 700), (40, 129, 2000), (300, 140, 260)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_matmul_bias_accumulate_and_stride(M, N, K, out):
    t = DTYPES[out]
    a, a64 = quantized(M, K, 1, 1)
    b, b64 = quantized(N, K, 128, 2)
    bias, base = random(1, N, t, 5)[0] * 1000, random(M, N, t, 6) * 1000
    store = torch.full((M, N + 3), 7.0, dtype=t, device="cuda")
    c = store[:, :N]
    c.copy_(base)
    got = fp8.matmul(a, b, bias=bias, out=c, accumulate=True)
    assert got is c and bool((store[:, N:] == 7).all())
    check_product(c, a64, b64, K, f64(bias), f64(base))
    check_product(fp8.matmul(a, b, bias=bias, out_dtype=t), a64, b64, K, f64(bias))


@pytest.mark.parametrize("M,N,K", [
    (2, 17, 128), (3, 33, 1543), (8, 16, 16), (7, 1, 100), (5, 2432, 4100), (8, 130, 8192), (4, 2433, 4224),
    (8, 8191, 300), (1, 8191, 2040), (2, 8193, 1100), (9, 200, 700), (1, 40, 20000)])
@pytest.mark.parametrize("out", sorted(DTYPES))
@pytest.mark.parametrize("blocks", [1, 128])
def test_matmul_of_few_tokens(M, N, K, out, blocks):
    """Both kernels that take few tokens, with blocks of either side's rows."""
    t = DTYPES[out]
    a, a64 = quantized(M, K, blocks, 1)
    b, b64 = quantized(N, K, 129 - blocks, 2)
    if out == "fp16":                                          # fp16 ends at 65504
        a64, b64 = a64 * 2.0 ** -12, b64 * 2.0 ** -8
        a.scales.view(torch.uint8).sub_(12)
        b.scales.view(torch.uint8).sub_(8)
    bias, base = random(1, N, t, 5)[0], random(M, N, t, 6)
    store = torch.full((M, N + 5), 7.0, dtype=t, device="cuda")
    c = store[:, :N]
    c.copy_(base)
    fp8.matmul(a, b, bias=bias, out=c, accumulate=True)
    check_product(c, a64, b64, K, f64(bias), f64(base))
    assert bool((store[:, N:] == 7).all())
    first = fp8.matmul(a, b, out_dtype=t)
    check_product(first, a64, b64, K)
    assert torch.equal(fp8.matmul(a, b, out_dtype=t), first)


@pytest.mark.parametrize("M", [1, 8])
def test_matmul_of_few_tokens_scales_and_nan(M):
    """Scales whose product leaves a float's range, that come back into it, and
    that are NaN; NaN and zeros in the values."""
    a, a64 = quantized(M, 512, 1, 1)
    b, b64 = quantized(5, 512, 1, 2)
    ea, eb = (torch.tensor(e) for e in ([-127, 127, 60, -60], [127, -127, -60, 60]))
    a.scales.view(torch.uint8).copy_((ea + 127).to(torch.uint8).expand(M, 4))
    b.scales.view(torch.uint8).copy_((eb + 127).to(torch.uint8).expand(5, 4))
    av, bv = f64(a.data), f64(b.data)
    check_product(fp8.matmul(a, b, out_dtype=torch.float32), av, bv, 512)
    a.scales.view(torch.uint8).fill_(1)                        # 2^-252 in all: nothing is left
    b.scales.view(torch.uint8).fill_(1)
    assert bool((fp8.matmul(a, b, out_dtype=torch.float32) == 0).all())
    b.scales.view(torch.uint8).fill_(253)                      # 2^0 again
    check_product(fp8.matmul(a, b, out_dtype=torch.float32), av, bv, 512)
    b.scales.view(torch.uint8)[2, 1] = 255
    b.data.view(torch.uint8)[3, 500] = 0x7f
    got = torch.isnan(fp8.matmul(a, b, out_dtype=torch.float32)).cpu()
    assert got[:, 2:4].all() and not got[:, :2].any() and not got[:, 4].any()


def test_matmul_of_128_row_blocks_on_both_sides():
    a, a64 = quantized(300, 400, 128, 1)
    b, b64 = quantized(200, 400, 128, 2)
    check_product(fp8.matmul(a, b, out_dtype=torch.float32), a64, b64, 400)


def test_matmul_repeats_bit_for_bit():
    a, _ = quantized(24, 4000, 1, 1)
    b, _ = quantized(500, 4000, 1, 2)
    first = fp8.matmul(a, b, out_dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(fp8.matmul(a, b, out_dtype=torch.float32), first)


def test_matmul_of_nothing():
    a, b = fp8.Quantized.empty(5, 0), fp8.Quantized.empty(7, 0)
    bias = torch.arange(7, dtype=torch.bfloat16, device="cuda")
    assert bool((fp8.matmul(a, b) == 0).all())
    assert torch.equal(fp8.matmul(a, b, bias=bias), bias.expand(5, 7))
    c = torch.ones(5, 7, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(fp8.matmul(a, b, bias=bias, out=c, accumulate=True), bias.expand(5, 7) + 1)
    assert fp8.matmul(fp8.Quantized.empty(0, 128), fp8.Quantized.empty(7, 128)).shape == (0, 7)


def test_matmul_nan_stays_in_its_row_and_column():
    a, a64 = quantized(40, 300, 1, 1)
    b, b64 = quantized(140, 300, 1, 2)
    a.data.view(torch.uint8)[3, 299] = 0x7F
    b.data.view(torch.uint8)[131, 0] = 0xFF
    c = fp8.matmul(a, b, out_dtype=torch.float32).cpu()
    bad = torch.isnan(c)
    assert bool(bad[3].all()) and bool(bad[:, 131].all()) and int(bad.sum()) == 140 + 40 - 1


def test_matmul_scales_at_their_ends():
    """Scale bytes 0 and 254 (2^-127 and 2^127) against each other."""
    a, _ = quantized(20, 128, 1, 1)
    b, _ = quantized(130, 128, 1, 2)
    plain = fp8.matmul(a, b, out_dtype=torch.float32)
    a.scales.view(torch.uint8).copy_(torch.full((20, 1), 0, dtype=torch.uint8))
    b.scales.view(torch.uint8).copy_(torch.full((130, 1), 254, dtype=torch.uint8))
    extreme = fp8.matmul(a, b, out_dtype=torch.float32)
    a.scales.view(torch.uint8).fill_(127)
    b.scales.view(torch.uint8).fill_(127)
    assert torch.equal(extreme, fp8.matmul(a, b, out_dtype=torch.float32))
    assert bool(torch.isfinite(plain).all())


def c_matrix(q):
    """A Quantized for the ctypes binding."""
    d, s = q.data, q.scales
    return basp.basp_fp8_matrix(d.data_ptr(), s.data_ptr(), *d.shape, d.stride(0), s.stride(0), q.block_rows)


def test_binding_and_tensors_give_the_same():
    """The ctypes binding's calls, with outputs of the caller's."""
    x, r, w = (random(n, 512, torch.bfloat16, i) for i, n in enumerate((40, 40, 1)))
    w, stream = w[0], torch.cuda.current_stream()
    y, h, rstd = fp8.rmsnorm(x, w, residual=r)
    q, h2, rstd2 = fp8.Quantized.empty(40, 512), torch.empty_like(x), torch.empty_like(rstd)
    basp.basp_rmsnorm(x, r, w, 1e-6, h=h2, q=c_matrix(q), rstd=rstd2, stream=stream)
    assert torch.equal(h, h2) and torch.equal(rstd, rstd2)
    assert torch.equal(q.data.view(torch.uint8), y.data.view(torch.uint8))
    wq = fp8.quantize(random(96, 512, torch.float32, 5), block_rows=128)
    c = torch.empty(40, 96, dtype=torch.bfloat16, device="cuda")
    basp.basp_matmul_fp8(c_matrix(q), c_matrix(wq), None, c, stream=stream)
    assert torch.equal(c, fp8.matmul(y, wq))
    dx, dw = torch.empty_like(x), torch.empty(512, device="cuda")
    ws = torch.empty(basp.basp_rmsnorm_backward_workspace(40, 512), dtype=torch.uint8, device="cuda")
    basp.basp_rmsnorm_backward(x, h, rstd, w, None, dx, dw, ws, stream=stream)
    want = fp8.rmsnorm_backward(x, h, rstd, w)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("how", ["dtype", "shape", "columns", "cpu", "bias", "scales", "out", "block_rows", "rows"])
def test_refusals(how):
    x, w = random(4, 256, torch.bfloat16, 1), torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, _ = quantized(4, 256, 1, 1)
    call = {
        "dtype": lambda: fp8.rmsnorm(x, w, residual=x.half()),
        "shape": lambda: fp8.rmsnorm(x, w[:255]),
        "columns": lambda: fp8.quantize(x.t()),
        "cpu": lambda: fp8.rmsnorm(x, w, residual=x.cpu()),
        "bias": lambda: fp8.matmul(q, q, bias=torch.zeros(4, device="cuda")),
        "scales": lambda: fp8.matmul(fp8.Quantized(q.data, q.scales[:, :1]), q),
        "out": lambda: fp8.matmul(q, q, out=torch.zeros(4, 5, dtype=torch.bfloat16, device="cuda")),
        "block_rows": lambda: fp8.matmul(fp8.Quantized(q.data, q.scales, 2), q),
        "rows": lambda: fp8.rmsnorm(torch.zeros(8, 4, 256, device="cuda")[::2, ::2], torch.ones(256, device="cuda"),
                                    residual=torch.zeros(4, 2, 256, device="cuda").transpose(0, 1).reshape(2, 4, 256)
                                    .transpose(0, 1)),
    }[how]
    with pytest.raises(ValueError):
        call()


def test_overlapping_output_is_refused():
    x = random(4, 256, torch.bfloat16, 1)
    with pytest.raises(basp.BaspError) as e:
        fp8.rmsnorm(x[:3], torch.ones(256, dtype=torch.bfloat16, device="cuda"), residual=x[:3].clone(), h=x[1:])
    assert e.value.status == basp.BASP_ERR_ALIASING


def test_scales_end_with_their_storage():
    """A last row of scales without the bytes up to a multiple of four."""
    q, q64 = quantized(5, 700, 1, 3)
    scales = torch.empty_strided((5, 6), (8, 1), dtype=torch.float8_e8m0fnu, device="cuda")
    scales.view(torch.uint8).copy_(q.scales.view(torch.uint8))
    assert scales.untyped_storage().nbytes() == 4 * 8 + 6
    b, b64 = quantized(9, 700, 128, 4)
    check_product(fp8.matmul(fp8.Quantized(q.data, scales), b, out_dtype=torch.float32), q64, b64, 700)


def test_other_stream_and_graph():
    """The calls follow the current stream, and a captured chain replays."""
    x, r = random(64, 2048, torch.bfloat16, 1), random(64, 2048, torch.bfloat16, 2)
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    wq, _ = quantized(512, 2048, 128, 3)

    def chain():
        q, h, _ = fp8.rmsnorm(x, w, residual=r)
        return h, fp8.matmul(q, wq)

    want = chain()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = chain()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    x.copy_(random(64, 2048, torch.bfloat16, 9))
    g.replay()
    want = chain()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_zz_no_wait_ran_out():
    assert basp.basp_matmul_fp8_timeouts() == 0
