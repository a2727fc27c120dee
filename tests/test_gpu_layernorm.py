"""The layer norm and its gradient (include/basp_fp8.h) against their 64-bit forms.

Tolerances.  u(t) = finfo(t).eps / 2 is one rounding to t; a 32-bit sum of n values has
n * 2^-24 of its sum of magnitudes.  The mean is off by em = (n + 2) 2^-24 mean|h|, a
deviation c = h - mean by that and a rounding of itself; the variance by 2 mean|c| em +
(n + 8) 2^-24 var, rstd by half of that of itself (relative) and 2^-24."""
import numpy as np
import pytest
import torch

import fp8_reference as ref8
import layer_reference as ref
from sequence_re_layout_gb300 import autograd, fp8

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F32, TINY = ref.F32, ref.TINY
SHAPES = [(1, 1), (1, 8), (1, 2048), (1, 2047), (3, 5000), (305, 64), (305, 63), (400, 1000), (400, 1001), (306, 4096),
          (310, 8192), (310, 8200), (2, 20001), (305, 16384), (305, 20000)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sequence_re_layout_gb300.build import build_library
    build_library()


def u(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def random(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).cuda()


def close(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= bound).all(), np.abs((got - want) / bound).max()


def forward_bounds(h, w, eps):
    """(mean's error, rstd's relative error, y's error before its own rounding)."""
    n = h.shape[1]
    em = (n + 2) * F32 * np.abs(h).mean(1)
    y, mean, rstd = ref.layernorm(h, w, None, eps)
    c = np.abs(h - mean[:, None])
    var = (c * c).mean(1)
    ev = 2 * c.mean(1) * (em + F32 * c.max(1)) + em * em + (n + 8) * F32 * var
    er = np.minimum(ev / (2 * (var + eps)) + 2 * F32, 1.0) + (ev / (var + eps)) ** 2
    ey = (rstd * (1 + er))[:, None] * (em[:, None] + F32 * c + c * (er[:, None] + 3 * F32)) * np.abs(w)
    return em, er, ey


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("residual,bias", [(True, True), (False, False), (True, False)])
def test_forward(rows, cols, dtype, residual, bias):
    t, eps = DTYPES[dtype], 1e-5
    wt = torch.float32 if rows % 2 else t
    x = random(rows, cols, dtype=t, seed=1, shift=0.5)
    r = random(rows, cols, dtype=t, seed=2) if residual else None
    w = random(cols, dtype=wt, seed=3)
    b = random(cols, dtype=wt, seed=4) if bias else None
    y, h, mean, rstd = fp8.layernorm(x, w, b, r, eps, quantized=False)
    h64 = f64(x + r) if residual else f64(x)
    assert np.array_equal(f64(h), h64) and y.dtype == h.dtype == t
    want, m, s = ref.layernorm(h64, f64(w), f64(b) if bias else None, eps)
    em, er, ey = forward_bounds(h64, f64(w), eps)
    close(mean, m, em + F32 * np.abs(m))
    close(rstd, s, (er + 2 * F32) * s)
    ey = ey + 2 * F32 * (np.abs(want) + (np.abs(f64(b)) if bias else 0))
    close(y, want, ey + u(t) * (np.abs(want) + ey) + TINY)
    q, h2, mean2, rstd2 = fp8.layernorm(x, w, b, r, eps)
    assert torch.equal(h, h2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    # the 8-bit values are within half a step (2^-4) of y where the scale is y's, or the next
    values, exps = ref8.quantize(want, 1)
    e = q.scales.cpu().view(torch.uint8).numpy().astype(np.int64) - 127
    assert (np.abs(e - exps) <= 1).all() and (e != exps).mean() <= 0.01
    scale = 2.0 ** e[:, np.arange(cols) // 128].astype(np.float64)
    got = f64(q.data.float()) * scale
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale + 1.0625 * ey).all()


def test_large_mean():
    """A mean a thousand times the deviation: sum(h^2) - mean^2 would lose every digit."""
    x = random(600, 1024, dtype=torch.float32, seed=1, shift=4096.0)
    w = torch.ones(1024, device="cuda")
    for rows in (600, 3):
        y, _, mean, rstd = fp8.layernorm(x[:rows], w, quantized=False)
        h = f64(x[:rows])
        want, m, s = ref.layernorm(h, np.ones(1024), None, 1e-5)
        em, er, ey = forward_bounds(h, np.ones(1024), 1e-5)
        close(mean, m, em)
        close(rstd, s, er * s)
        close(y, want, ey + 2 * F32 * np.abs(want))
        assert np.abs(f64(rstd) / s - 1).max() < 1e-4


@pytest.mark.parametrize("rows,cols", [(1, 128), (400, 256), (4, 5000), (400, 129)])
def test_values_that_are_no_numbers(rows, cols):
    """A NaN or an infinity stays in its row; constant rows have rstd = eps^-1/2."""
    x = random(rows, cols, dtype=torch.float32, seed=1)
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    want = fp8.layernorm(x, w, b, quantized=False)
    for bad in (float("nan"), float("inf")):
        z = x.clone()
        z[0, cols // 2] = bad
        y, _, mean, rstd = fp8.layernorm(z, w, b, quantized=False)
        assert bool(torch.isnan(rstd[0])) and bool(torch.isnan(y[0]).all()) and torch.equal(y[1:], want[0][1:])
        q = fp8.layernorm(z, w, b)[0]
        assert bool(torch.isnan(q.data[0].float()).all())
    y, _, mean, rstd = fp8.layernorm(torch.full_like(x, 3.0), w, b, quantized=False)
    assert bool((y == 0).all()) and bool((mean == 3).all()) and np.abs(f64(rstd) - 1e-5 ** -0.5).max() < 1e-4


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("dh", [True, False])
def test_backward(rows, cols, dtype, dh):
    t = DTYPES[dtype]
    h, dy = random(rows, cols, dtype=t, seed=1, shift=0.5), random(rows, cols, dtype=t, seed=2)
    d = random(rows, cols, dtype=t, seed=3) if dh else None
    w = random(cols, dtype=torch.float32 if rows % 2 else t, seed=4)
    _, _, mean, rstd = fp8.layernorm(h, w, quantized=False)
    dx, dw, db = fp8.layernorm_backward(dy, h, mean, rstd, w, d)
    check_backward(dx, dw, db, dy, h, mean, rstd, w, d, t)
    assert torch.equal(fp8.layernorm_backward(dy, h, mean, rstd, w, d, need_dbias=False)[1], dw)
    part = fp8.layernorm_backward(dy, h, mean, rstd, w, d, need_dweight=False)
    assert part[1] is None and torch.equal(part[2], db) and torch.equal(part[0], dx)
    none = fp8.layernorm_backward(dy, h, mean, rstd, w, d, False, False)
    assert none[1] is None and none[2] is None and torch.equal(none[0], dx)


def check_backward(dx, dw, db, dy, h, mean, rstd, w, d, t, wt=torch.float32):
    """The bound for the mean and rstd as they were given."""
    h64, g64, m, s, w64 = (f64(x) for x in (h, dy, mean, rstd, w))
    rows, cols = h64.shape
    rx, rw, rb = ref.layernorm_backward(g64, h64, m, s, w64, f64(d) if d is not None else None)
    n, g = np.abs((h64 - m[:, None]) * s[:, None]), np.abs(g64 * w64)
    size = s[:, None] * (g + g.mean(1, keepdims=True) + n * (g * n).mean(1, keepdims=True))
    bx = (2 * cols + 32) * F32 * size + 2 * F32 * (np.abs(f64(d)) if d is not None else 0)
    close(dx, rx, bx + u(t) * (np.abs(rx) + bx) + TINY)
    close(dw, rw, (rows + 8) * F32 * (np.abs(g64) * n).sum(0) + u(wt) * np.abs(rw) + TINY)
    close(db, rb, (rows + 8) * F32 * np.abs(g64).sum(0) + u(wt) * np.abs(rb) + TINY)


@pytest.mark.parametrize("rows,cols", [(5, 256), (700, 1000), (700, 333)])
def test_strides_and_places(rows, cols):
    """Rows apart from each other, h written over x or the residual, dx over dy or dh's place left alone."""
    t = torch.bfloat16
    wide = random(rows, cols + 24, dtype=t, seed=1)
    x, r = wide[:, 8:8 + cols], random(rows, 2 * cols, dtype=t, seed=2)[:, :cols]
    w, b = random(cols, dtype=t, seed=3), random(cols, dtype=t, seed=4)
    want = fp8.layernorm(x.contiguous(), w, b, r.contiguous(), quantized=False)
    for got in (fp8.layernorm(x, w, b, r, quantized=False), fp8.layernorm(x, w, b, r.clone(), quantized=False)):
        close(got[0], f64(want[0]), 2 * u(t) * np.abs(f64(want[0])) + 2.0 ** -12)
        assert torch.equal(got[1], want[1])
    over = x.clone()
    y, h, _, _ = fp8.layernorm(over, w, b, r.contiguous(), quantized=False, h=over)
    assert h is over and torch.equal(over, want[1]) and torch.equal(y, want[0])
    edge = wide.clone()
    fp8.layernorm(edge[:, 8:8 + cols], w, b, r, h=edge[:, 8:8 + cols])
    assert torch.equal(edge[:, :8], wide[:, :8]) and torch.equal(edge[:, 8 + cols:], wide[:, 8 + cols:])


def test_sizes_of_zero():
    for t in DTYPES.values():
        w = torch.ones(64, dtype=t, device="cuda")
        y, h, mean, rstd = fp8.layernorm(torch.empty(0, 64, dtype=t, device="cuda"), w)
        assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
        y, h, mean, rstd = fp8.layernorm(torch.empty(7, 0, dtype=t, device="cuda"), w[:0], quantized=False)
        assert y.shape == (7, 0) and bool(torch.isnan(mean).all()) and bool(torch.isnan(rstd).all())
        e = torch.empty(0, 64, dtype=t, device="cuda")
        dx, dw, db = fp8.layernorm_backward(e, e, mean[:0], rstd[:0], w)
        assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
        e = torch.empty(7, 0, dtype=t, device="cuda")
        dx, dw, db = fp8.layernorm_backward(e, e, mean, rstd, w[:0])
        assert dx.shape == (7, 0) and dw.shape == db.shape == (0,)


def test_many_rows_repeat():
    x, w = random(20000, 512, dtype=torch.bfloat16, seed=1), random(512, dtype=torch.bfloat16, seed=2)
    dy = random(20000, 512, dtype=torch.bfloat16, seed=3)
    y, h, mean, rstd = fp8.layernorm(x, w, quantized=False)
    want = fp8.layernorm_backward(dy, h, mean, rstd, w)
    for _ in range(3):
        assert torch.equal(fp8.layernorm(x, w, quantized=False)[0], y)
        assert all(torch.equal(a, b) for a, b in zip(fp8.layernorm_backward(dy, h, mean, rstd, w), want))
    check_backward(*want, dy, h, mean, rstd, w, None, torch.bfloat16)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("through", ["y", "h", "both"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_autograd(residual, bias, through, dtype):
    t, rows, cols = DTYPES[dtype], 310, 257
    x = random(rows, cols, dtype=t, seed=1).requires_grad_()
    r = random(rows, cols, dtype=t, seed=2).requires_grad_() if residual else None
    w = random(cols, dtype=t, seed=3).requires_grad_()
    b = random(cols, dtype=t, seed=4).requires_grad_() if bias else None
    dy, dh = random(rows, cols, dtype=t, seed=5), random(rows, cols, dtype=t, seed=6)
    y, h = autograd.layernorm(x, w, b, r)
    outs = {"y": [(y, dy)], "h": [(h, dh)], "both": [(y, dy), (h, dh)]}[through]
    torch.autograd.backward([o for o, _ in outs], [d for _, d in outs])
    y2, h2, mean, rstd = fp8.layernorm(x.detach(), w.detach(), None if b is None else b.detach(),
                                       None if r is None else r.detach(), quantized=False)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    if through == "h":
        assert torch.equal(x.grad, dh) and w.grad is None
    else:
        dx, dw, db = fp8.layernorm_backward(dy, h2, mean, rstd, w.detach(), dh if through == "both" else None)
        assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw.to(t))
        assert not bias or torch.equal(b.grad, db.to(t))
    assert not residual or torch.equal(r.grad, x.grad)


def test_gradient_against_differences():
    """Central differences of the 64-bit form (step 2^-12: off by its square times a
    third derivative of order one, and by 2^-52 / 2^-12 of the values)."""
    rows, cols, step = 7, 130, 2.0 ** -12
    x = random(rows, cols, dtype=torch.float32, seed=1).requires_grad_()
    w, b = (random(cols, dtype=torch.float32, seed=s).requires_grad_() for s in (2, 3))
    dy, dh = random(rows, cols, dtype=torch.float32, seed=4), random(rows, cols, dtype=torch.float32, seed=5)
    torch.autograd.backward(autograd.layernorm(x, w, b), [dy, dh])
    vx = np.random.default_rng(6).standard_normal((rows, cols))
    vw, vb = (np.random.default_rng(s).standard_normal(cols) for s in (7, 8))

    def value(s):
        h = f64(x) + s * vx
        return (f64(dy) * ref.layernorm(h, f64(w) + s * vw, f64(b) + s * vb, 1e-5)[0]).sum() + (f64(dh) * h).sum()

    want = (value(step) - value(-step)) / (2 * step)
    terms = [f64(x.grad) * vx, f64(w.grad) * vw, f64(b.grad) * vb]
    size = sum(np.abs(t).sum() for t in terms)
    assert abs(sum(t.sum() for t in terms) - want) <= (8 * cols * F32 + 2.0 ** -18) * size


@pytest.mark.parametrize("residual", [False, True])
def test_linear(residual):
    """The norm and the projection of its result: what the two calls give one after the other."""
    t, rows, cols, n_out = torch.bfloat16, 150, 384, 260
    x = random(rows, cols, dtype=t, seed=1).requires_grad_()
    r = random(rows, cols, dtype=t, seed=2).requires_grad_() if residual else None
    nw, nb = random(cols, dtype=t, seed=3).requires_grad_(), random(cols, dtype=t, seed=4).requires_grad_()
    w = random(n_out, cols, dtype=torch.float32, seed=5, scale=cols ** -0.5).requires_grad_()
    b = random(n_out, dtype=t, seed=6).requires_grad_()
    dy, dh = random(rows, n_out, dtype=t, seed=7), random(rows, cols, dtype=t, seed=8)
    y, h = autograd.layernorm_linear_fp8(x, nw, nb, w, b, r)
    torch.autograd.backward([y, h], [dy, dh])
    leaves = [None if p is None else p.detach() for p in (x, nw, nb, r)]
    q, h2, mean, rstd = fp8.layernorm(*leaves)
    w8, w8t = fp8.quantize(w.detach(), block_rows=128, transposed=True)
    assert torch.equal(h, h2) and torch.equal(y, fp8.matmul(q, w8, bias=b.detach()))
    d8, d8t = fp8.quantize(dy, transposed=True)
    dn = fp8.matmul(d8, w8t)
    dx, dnw, dnb = fp8.layernorm_backward(dn, h2, mean, rstd, nw.detach(), dh)
    assert torch.equal(x.grad, dx) and torch.equal(nw.grad, dnw.to(t)) and torch.equal(nb.grad, dnb.to(t))
    n16 = fp8.layernorm(h2, nw.detach(), nb.detach(), quantized=False)[0]
    x8t = fp8.quantize(n16, rows=False, transposed=True)
    assert torch.equal(w.grad, fp8.matmul(d8t, x8t, out_dtype=torch.float32))
    assert torch.equal(b.grad, dy.sum(0, dtype=torch.float32).to(t))
    assert not residual or torch.equal(r.grad, x.grad)
    with torch.no_grad():
        again = autograd.layernorm_linear_fp8(x, nw, nb, w8, b, r)
    assert torch.equal(again[0], y) and torch.equal(again[1], h)


def test_captured():
    x, w, dy = (random(*s, dtype=torch.bfloat16, seed=i) for i, s in enumerate(((900, 256), (256,), (900, 256))))
    def run():
        y, h, mean, rstd = fp8.layernorm(x, w, quantized=False)
        return (y, mean, rstd, *fp8.layernorm_backward(dy, h, mean, rstd, w))
    want = run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("cols", [257, 385, 1001, 2047, 4095, 5003, 6143, 8191])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_warps_of_a_row_that_differ(cols, dtype):
    """Warps whose blocks all end inside the row read without checks, the others with; they
    meet at one barrier, in each of more rows than there are CTAs."""
    t, rows = DTYPES[dtype], 1300
    h, dy, d = (random(rows, cols, dtype=t, seed=s) for s in (1, 2, 3))
    w = random(cols, dtype=torch.float32, seed=4)
    _, _, mean, rstd = fp8.layernorm(h, w, quantized=False)
    got = fp8.layernorm_backward(dy, h, mean, rstd, w, d)
    check_backward(*got, dy, h, mean, rstd, w, d, t)
    assert all(torch.equal(a, b) for a, b in zip(got, fp8.layernorm_backward(dy, h, mean, rstd, w, d)))
