"""The differentiable 8-bit projections (autograd.py) and the attention layer
they make with the re-layout (examples/attention_layer.py), against plain
64-bit forms.

Tolerances.  u(t) = finfo(t).eps / 2 is one rounding to t.  The 8-bit operands
themselves are known exactly (tests/fp8_reference.py rounds them), so a product
has at most 2^-23 of its sum of magnitudes for each 32 terms, and the rounding
of its result; a 32-bit sum of n values has n * 2^-24 of its sum of magnitudes.
Where a result passes through a second operator, the first one's bound goes
through that operator's derivative."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp8_reference as ref
import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import autograd, fp8

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F32 = 2.0 ** -24
TINY = 2.0 ** -25                       # the last step of fp16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sequence_re_layout_gb300.build import build_library
    build_library()


def u(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def random(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def rounded(x, block_rows=1):
    """What x stands for once it is rounded to 8 bits."""
    return ref.dequantize(*ref.quantize(x, block_rows), block_rows)


def product(a, b, dtype):
    """(a b^T, bound of the operator's error) of exactly known operands."""
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    return want, u(dtype) * np.abs(want) + (-(-a.shape[1] // 32) + 16) * 2.0 ** -23 * size + TINY


def close(got, want, bound):
    assert (np.abs(f64(got) - want) <= bound).all(), np.abs((f64(got) - want) / bound).max()


@pytest.mark.parametrize("rows,n_in,n_out", [(1, 128, 64), (3, 200, 129), (130, 256, 384), (300, 77, 515)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("master", [False, True])
def test_linear(rows, n_in, n_out, dtype, master):
    t, wt = DTYPES[dtype], torch.float32 if master else DTYPES[dtype]
    x = random(rows, n_in, dtype=t, seed=1).requires_grad_()
    w = random(n_out, n_in, dtype=wt, seed=2, scale=n_in ** -0.5).requires_grad_()
    b = random(n_out, dtype=t, seed=3).requires_grad_()
    dy = random(rows, n_out, dtype=t, seed=4)
    y = autograd.linear_fp8(x, w, b)
    y.backward(dy)
    assert y.dtype == t and x.grad.dtype == t and w.grad.dtype == wt and b.grad.dtype == t
    x64, w64, d64 = f64(x), f64(w), f64(dy)
    want, bound = product(rounded(x64), rounded(w64, 128), t)
    close(y, want + f64(b), bound + (u(t) + 2.0 ** -23) * np.abs(f64(b)))
    close(x.grad, *product(rounded(d64), rounded(w64, 128).T, t))
    close(w.grad, *product(rounded(d64.T), rounded(x64.T), wt))
    db = d64.sum(0)
    close(b.grad, db, u(t) * np.abs(db) + (rows + 8) * F32 * np.abs(d64).sum(0) + TINY)


def test_linear_keeps_only_what_its_gradients_need():
    """Any subset of the inputs may want a gradient, with the same results."""
    x, w = random(70, 200, dtype=torch.bfloat16, seed=1), random(90, 200, dtype=torch.float32, seed=2)
    b, dy = random(90, dtype=torch.bfloat16, seed=3), random(70, 90, dtype=torch.bfloat16, seed=4)
    full = [t.clone().requires_grad_() for t in (x, w, b)]
    y = autograd.linear_fp8(*full)
    y.backward(dy)
    for want in range(1, 8):
        leaves = [t.clone().requires_grad_(bool(want >> i & 1)) for i, t in enumerate((x, w, b))]
        got = autograd.linear_fp8(*leaves)
        got.backward(dy)
        assert torch.equal(got, y)
        for i, (a, f) in enumerate(zip(leaves, full)):
            assert torch.equal(a.grad, f.grad) if want >> i & 1 else a.grad is None
    with torch.no_grad():
        assert torch.equal(autograd.linear_fp8(x, w, b), y)
        assert torch.equal(autograd.linear_fp8(x, fp8.quantize(w, block_rows=128), b), y)


def test_linear_shapes():
    """Leading dimensions, one row without any, strided rows, a gradient that is
    one value spread over the result, and no rows."""
    w = random(48, 96, dtype=torch.bfloat16, seed=2).requires_grad_()
    x = random(6, 96, dtype=torch.bfloat16, seed=1)
    y = autograd.linear_fp8(x, w)
    assert torch.equal(autograd.linear_fp8(x.view(2, 3, 96), w), y.view(2, 3, 48))
    assert torch.equal(autograd.linear_fp8(x[2], w), y[2])
    wide = torch.full((6, 160), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 32:128] = x
    assert torch.equal(autograd.linear_fp8(wide[:, 32:128], w), y)
    xg = x.view(2, 3, 96).clone().requires_grad_()
    autograd.linear_fp8(xg, w).sum().backward()
    close(xg.grad.view(6, 96), *product(np.ones((6, 48)), rounded(f64(w), 128).T, torch.bfloat16))
    none = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w.grad = None
    y = autograd.linear_fp8(none, w)
    y.backward(torch.empty_like(y))
    assert y.shape == (0, 48) and none.grad.shape == (0, 96) and bool((w.grad == 0).all())


def norm_bounds(dy, dy_error, h, rstd, w, dh, t):
    """(dx, bound, dweight, bound) of the norm's backward, with dy off by dy_error."""
    rx, rw = ref.norm_backward(dy, h, rstd, w, dh)
    cols, n = h.shape[1], np.abs(h * rstd[:, None])
    def through(d):
        g = np.abs(d * w)
        return rstd[:, None] * (g + n * (g * n).mean(1, keepdims=True))
    size = through(np.abs(dy) + dy_error) + (0 if dh is None else np.abs(dh))
    bx = u(t) * np.abs(rx) + (2 * cols + 32) * F32 * size + (1 + u(t)) * through(dy_error) + TINY
    sw = ((np.abs(dy) + dy_error) * n).sum(0)
    bw = (h.shape[0] + cols + 32) * F32 * sw + (np.abs(dy_error) * n).sum(0)
    return rx, bx, rw, bw


@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 129), (300, 256), (40, 1000)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("grads", ["y", "h", "both"])
def test_rmsnorm(rows, cols, dtype, residual, grads):
    t = DTYPES[dtype]
    x = random(rows, cols, dtype=t, seed=1).requires_grad_()
    r = random(rows, cols, dtype=t, seed=2).requires_grad_() if residual else None
    w = random(cols, dtype=torch.float32 if rows % 2 else t, seed=3).requires_grad_()
    dy, dh = random(rows, cols, dtype=t, seed=4), random(rows, cols, dtype=t, seed=5)
    y, h = autograd.rmsnorm(x, w, r)
    torch.autograd.backward([y, h] if grads == "both" else [y] if grads == "y" else [h],
                            [dy, dh] if grads == "both" else [dy] if grads == "y" else [dh])
    h64 = f64(x + r) if residual else f64(x)
    assert np.array_equal(f64(h), h64)
    want, rstd = ref.norm(h64, f64(w), 1e-6)
    close(y, want, u(t) * np.abs(want) + (cols / 2 + 8) * F32 * np.abs(want) + TINY)
    if residual:
        assert torch.equal(r.grad, x.grad)
    if grads == "h":
        assert torch.equal(x.grad, dh) and w.grad is None
        return
    rx, bx, rw, bw = norm_bounds(f64(dy), np.zeros((rows, cols)), h64, rstd, f64(w), f64(dh) if grads == "both" else None, t)
    close(x.grad, rx, bx)
    close(w.grad, rw, bw + u(w.dtype) * np.abs(rw) + TINY)


def test_rmsnorm_gradient_against_differences():
    """The directional derivative of sum(dy y + dh h), by central differences of
    the 64-bit form (step 2^-12: off by its square times a third derivative of
    order one, and by 2^-52 / 2^-12 of the values)."""
    rows, cols, step = 7, 130, 2.0 ** -12
    x, r = (random(rows, cols, dtype=torch.float32, seed=s).requires_grad_() for s in (1, 2))
    w = random(cols, dtype=torch.float32, seed=3).requires_grad_()
    dy, dh = random(rows, cols, dtype=torch.float32, seed=4), random(rows, cols, dtype=torch.float32, seed=5)
    torch.autograd.backward(autograd.rmsnorm(x, w, r), [dy, dh])
    vx, vr = (np.random.default_rng(s).standard_normal((rows, cols)) for s in (6, 7))
    vw = np.random.default_rng(8).standard_normal(cols)

    def value(s):
        h = f64(x) + s * vx + f64(r) + s * vr
        return (f64(dy) * ref.norm(h, f64(w) + s * vw, 1e-6)[0]).sum() + (f64(dh) * h).sum()

    want = (value(step) - value(-step)) / (2 * step)
    terms = [f64(x.grad) * vx, f64(r.grad) * vr, f64(w.grad) * vw]
    size = sum(np.abs(t).sum() for t in terms)
    assert abs(sum(t.sum() for t in terms) - want) <= (8 * cols * F32 + 2.0 ** -18) * size


def test_inputs_used_twice():
    """x that is its own residual, and one weight for two norms: the gradients add."""
    rows, cols, t = 33, 257, torch.float32
    x, w = random(rows, cols, dtype=t, seed=1).requires_grad_(), random(cols, dtype=t, seed=2).requires_grad_()
    d1, d2 = random(rows, cols, dtype=t, seed=3), random(rows, cols, dtype=t, seed=4)
    y1, h = autograd.rmsnorm(x, w, x)
    y2, _ = autograd.rmsnorm(h, w)
    torch.autograd.backward([y1, y2], [d1, d2])
    h64 = 2 * f64(x)
    rstd = ref.norm(h64, f64(w), 1e-6)[1]
    zero = np.zeros((rows, cols))
    r1, b1, w1, bw1 = norm_bounds(f64(d1), zero, h64, rstd, f64(w), None, t)
    r2, b2, w2, bw2 = norm_bounds(f64(d2), zero, h64, rstd, f64(w), None, t)
    close(x.grad, 2 * (r1 + r2), 2 * (b1 + b2) + 4 * F32 * np.abs(r1 + r2))
    close(w.grad, w1 + w2, bw1 + bw2 + 2 * F32 * np.abs(w1 + w2))


@pytest.mark.parametrize("rows,cols,n_out", [(1, 128, 64), (5, 200, 129), (150, 384, 260)])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("through_h", [False, True])
def test_rmsnorm_linear(rows, cols, n_out, dtype, residual, through_h):
    t = DTYPES[dtype]
    x = random(rows, cols, dtype=t, seed=1).requires_grad_()
    r = random(rows, cols, dtype=t, seed=2).requires_grad_() if residual else None
    nw = random(cols, dtype=t, seed=3).requires_grad_()
    w = random(n_out, cols, dtype=torch.float32, seed=4, scale=cols ** -0.5).requires_grad_()
    b = random(n_out, dtype=t, seed=5).requires_grad_()
    dy, dh = random(rows, n_out, dtype=t, seed=6), random(rows, cols, dtype=t, seed=7)
    y, h = autograd.rmsnorm_linear_fp8(x, nw, w, b, r)
    torch.autograd.backward([y, h] if through_h else [y], [dy, dh] if through_h else [dy])
    # the operands in 8 bits, as the norm itself gives them (tests/test_gpu_fp8.py holds it to the 64-bit form)
    q, h_, rstd = fp8.rmsnorm(x.detach(), nw.detach(), None if r is None else r.detach())
    y16 = fp8.rmsnorm(h_, nw.detach(), quantized=False)[0]
    assert torch.equal(h, h_)
    q64 = ref.dequantize(f64(q.data.float()), q.scales.cpu().view(torch.uint8).numpy().astype(np.int64) - 127, 1)
    w64, d64, b64 = rounded(f64(w), 128), f64(dy), f64(b)
    want, bound = product(q64, w64, t)
    close(y, want + b64, bound + (u(t) + 2.0 ** -23) * np.abs(b64))
    close(w.grad, *product(rounded(d64.T), rounded(f64(y16).T), torch.float32))
    db = d64.sum(0)
    close(b.grad, db, u(t) * np.abs(db) + (rows + 8) * F32 * np.abs(d64).sum(0) + TINY)
    dn, dn_error = product(rounded(d64), w64.T, t)
    rx, bx, rw, bw = norm_bounds(dn, dn_error, f64(h_), f64(rstd), f64(nw), f64(dh) if through_h else None, t)
    close(x.grad, rx, bx)
    close(nw.grad, rw, bw + u(t) * np.abs(rw) + TINY)
    if residual:
        assert torch.equal(r.grad, x.grad)


def test_rmsnorm_linear_keeps_only_what_its_gradients_need():
    x, r = (random(40, 256, dtype=torch.bfloat16, seed=s) for s in (1, 2))
    nw, w = random(256, dtype=torch.bfloat16, seed=3), random(100, 256, dtype=torch.bfloat16, seed=4)
    b, dy = random(100, dtype=torch.bfloat16, seed=5), random(40, 100, dtype=torch.bfloat16, seed=6)
    inputs = (x, nw, w, b, r)
    full = [t.clone().requires_grad_() for t in inputs]
    y, h = autograd.rmsnorm_linear_fp8(*full)
    y.backward(dy)
    for want in (1, 2, 4, 8, 16, 17, 12, 6):
        leaves = [t.clone().requires_grad_(bool(want >> i & 1)) for i, t in enumerate(inputs)]
        got, got_h = autograd.rmsnorm_linear_fp8(*leaves)
        got.backward(dy)
        assert torch.equal(got, y) and torch.equal(got_h, h)
        for i, (a, f) in enumerate(zip(leaves, full)):
            assert torch.equal(a.grad, f.grad) if want >> i & 1 else a.grad is None
    with torch.no_grad():
        for weight in (w, fp8.quantize(w, block_rows=128)):
            got, got_h = autograd.rmsnorm_linear_fp8(x, nw, weight, b, r)
            assert torch.equal(got, y) and torch.equal(got_h, h)


def test_second_derivatives_are_refused():
    x = random(4, 128, dtype=torch.float32, seed=1).requires_grad_()
    w = random(8, 128, dtype=torch.float32, seed=2).requires_grad_()
    g, = torch.autograd.grad(autograd.linear_fp8(x, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="does not require grad"):
        g.sum().backward()
    dy = random(4, 8, dtype=torch.float32, seed=3).requires_grad_()
    g, = torch.autograd.grad(autograd.linear_fp8(x, w), x, dy, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


def test_training_step_in_a_graph():
    """Forward and backward captured together, with no eager graph of the same
    leaves alive, replay on new inputs to what eager calls give."""
    x = random(64, 256, dtype=torch.bfloat16, seed=1).requires_grad_()
    nw = random(256, dtype=torch.bfloat16, seed=2).requires_grad_()
    w = random(384, 256, dtype=torch.float32, seed=3).requires_grad_()
    dy = random(64, 384, dtype=torch.bfloat16, seed=4)

    def step(leaves):
        y, _ = autograd.rmsnorm_linear_fp8(*leaves)
        return torch.autograd.grad(y, leaves, dy)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step((x, nw, w))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step((x, nw, w))
    with torch.no_grad():
        x.copy_(random(64, 256, dtype=torch.bfloat16, seed=8))
    graph.replay()
    torch.cuda.synchronize()
    eager = step([t.detach().clone().requires_grad_() for t in (x, nw, w)])
    assert all(torch.equal(a, b) for a, b in zip(captured, eager))


# ---- the layer ----------------------------------------------------------------

def example():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_layer(layer, x, residual, B, S):
    """The layer on full-precision leaves, in 64 bits on sequences in order."""
    i = layer.layout.info
    leaves = [p.detach().double().requires_grad_() for p in (layer.norm, layer.wqkv, layer.bqkv, layer.wo)]
    nw, wqkv, bqkv, wo = leaves
    h = (x + residual).double()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * nw
    qkv = (y @ wqkv.T + bqkv).view(B, S, -1, i["d"])
    q, k, v = (t.transpose(1, 2) for t in qkv.split([i["Hq"], i["Hkv"], i["Hkv"]], dim=2))
    k, v = (t.repeat_interleave(i["Hq"] // i["Hkv"], 1) for t in (k, v))
    mask = torch.ones(S, S, dtype=torch.bool, device="cuda").tril()
    p = torch.softmax((q @ k.transpose(-1, -2) * i["d"] ** -0.5).masked_fill(~mask, float("-inf")), -1)
    o = (p @ v).transpose(1, 2).reshape(B, S, -1)
    return o @ wo.T, h, leaves


@pytest.mark.parametrize("K", [2, 4])
def test_attention_layer(K):
    """Rounding an operand to 8 bits moves each value by at most 2^-4 of itself,
    independently: a product of two moves by at most 2^-4 sqrt(2) = 0.09 of
    itself in the mean square.  The layer's V and output products give that each;
    the scores (of order one) move by 0.09 sqrt(2) and the probabilities by as
    much of themselves: 0.18 in all.  The gradients pass one or two products
    more: below 0.35, a cosine above 0.9."""
    B, S, Hq, Hkv, d, N = 2, 256, 8, 4, 64, 4
    torch.manual_seed(1)
    with basp.Layout(B, S, Hq, Hkv, d, N, K, "bf16") as L:
        layer = example().AttentionLayer(L, Hq * d)
        bg, per = B // (N // K), S // K
        shards = lambda t: t.view(N // K, bg, K, per, -1).transpose(1, 2).reshape(B * S, -1)     # noqa: E731
        whole = lambda t: t.view(N // K, K, bg, per, -1).transpose(1, 2).reshape(B, S, -1)       # noqa: E731
        x, r = (torch.randn(B, S, Hq * d, device="cuda").bfloat16() for _ in range(2))
        dy = torch.randn(B, S, Hq * d, device="cuda").bfloat16()
        out, h = layer(shards(x), shards(r))
        want, want_h, leaves = plain_layer(layer, x, r, B, S)
        error = whole(out.detach()).double() - want.detach()
        assert float(error.norm() / want.detach().norm()) <= 0.2
        assert torch.equal(whole(h), (x + r))
        out.backward(shards(dy))
        want.backward(dy.double())
        for p, leaf in zip((layer.norm, layer.wqkv, layer.bqkv, layer.wo), leaves):
            assert float(torch.nn.functional.cosine_similarity(p.grad.double().flatten(), leaf.grad.flatten(), 0)) >= 0.9
        layer.freeze()
        with torch.no_grad():
            again, _ = layer(shards(x), shards(r))
        assert torch.equal(again, out)


def test_example_program():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "attention_layer.py"), "--seq", "512", "--steps", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split()[-1]) for line in r.stdout.splitlines() if "loss" in line]
    assert len(losses) == 3 and all(np.isfinite(losses)), r.stdout


def test_zz_no_wait_ran_out():
    assert basp.basp_matmul_fp8_timeouts() == 0
