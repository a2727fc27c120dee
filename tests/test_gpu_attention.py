"""Attention with a window and sinks (include/basp_attention.h) against its 64-bit
form; tests/layer_reference.py derives the bounds."""
import numpy as np
import pytest
import torch

import sequence_re_layout_gb300 as basp
from layer_reference import Attention, gradients_in_units
from sequence_re_layout_gb300 import attention, autograd

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def close(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), np.abs((got - want) / bound).max()


def check(q, k, v, do=None, window=None, sinks=0, scale=None):
    """Forward, and with `do` backward, of every sequence against 64 bits."""
    t, d = q.dtype, q.shape[3]
    o, lse = attention.forward(q, k, v, window, sinks, scale)
    grads = None if do is None else attention.backward(do, q, k, v, o, lse, window, sinks, scale)
    assert o.shape == q.shape and o.dtype == t and lse.shape == (q.shape[0], q.shape[2], q.shape[1])
    for b in range(q.shape[0]):
        r = Attention(f64(q[b]), f64(k[b]), f64(v[b]), window, sinks, d ** -0.5 if scale is None else scale, u(t))
        close(o[b], r.o, r.o_bound)
        some = np.isfinite(r.lse)
        got = f64(lse[b])
        assert np.array_equal(np.isneginf(got), ~some)
        assert (np.abs(got - r.lse)[some] <= r.lse_bound[some]).all()
        if do is not None:
            want, bound = r.backward(f64(do[b]), r.o_bound)
            for name, g in zip(("dq", "dk", "dv"), grads):
                close(g[b], want[name], bound[name])
    return o, lse, grads


def tensors(B, Sq, Sk, Hq, Hkv, d, t):
    return (random(B, Sq, Hq, d, dtype=t, seed=1), random(B, Sk, Hkv, d, dtype=t, seed=2),
            random(B, Sk, Hkv, d, dtype=t, seed=3), random(B, Sq, Hq, d, dtype=t, seed=4))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("Sq,Sk", [(1, 1), (2, 2), (64, 64), (127, 127), (128, 128), (129, 129), (257, 257), (300, 300),
                                   (1, 200), (77, 333), (130, 513), (5, 3), (200, 64), (3, 0)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (64, 4), (130, 0), (200, 150), (1000, 3), (33, 1000)])
def test_lengths_and_masks(Sq, Sk, window, sinks, dtype):
    q, k, v, do = tensors(1, Sq, Sk, 2, 1, 64, DTYPES[dtype])
    check(q, k, v, do, window, sinks)


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
@pytest.mark.parametrize("S", [70, 200, 400])
def test_head_sizes(S, d, dtype):
    q, k, v, do = tensors(1, S, S, 2, 2, d, DTYPES[dtype])
    check(q, k, v, do, 150, 4)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (4, 2), (6, 2), (8, 1), (5, 5)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_heads(Hq, Hkv, d):
    q, k, v, do = tensors(2, 261, 261, Hq, Hkv, d, torch.bfloat16)
    check(q, k, v, do, 140, 5)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 4.0])
def test_scales(scale):
    q, k, v, do = tensors(1, 190, 190, 2, 2, 64, torch.float16)
    check(q, k, v, do, 100, 2, scale)


@pytest.mark.parametrize("Sq,Sk,Hq,Hkv,d,window,sinks", [(4000, 4000, 2, 1, 64, 100, 3), (4000, 4000, 1, 1, 128, 300, 200),
                                                         (3001, 3001, 4, 2, 40, None, 0), (2500, 3000, 3, 1, 72, 64, 700)])
def test_long_key_tiles_are_shared(Sq, Sk, Hq, Hkv, d, window, sinks):
    """Few heads and many queries of the first keys: several CTAs share a tile of keys."""
    q, k, v, do = tensors(1, Sq, Sk, Hq, Hkv, d, torch.bfloat16)
    o, lse, g = check(q, k, v, do, window, sinks)
    assert all(torch.equal(a, b) for a, b in zip(g, attention.backward(do, q, k, v, o, lse, window, sinks)))
    bad = do.clone()
    bad[0, Sq - 1, 0, 3] = float("nan")
    r = Attention(*(f64(x)[0] for x in (q, k, v)), window, sinks, d ** -0.5, u(torch.bfloat16))
    want, bound = r.backward(f64(do)[0], r.o_bound)
    rows = ~r.sees[Sq - 1]
    got = attention.backward(bad, q, k, v, o, lse, window, sinks)
    for name, x in zip(("dk", "dv"), got[1:]):
        close(x[0][torch.from_numpy(rows).cuda()], want[name][rows], bound[name][rows])


def test_growing_scores():
    """A row's largest score grows from tile to tile by far more than 8 in the exponent of 2."""
    t, S, d = torch.bfloat16, 640, 64
    q, k, v, do = tensors(1, S, S, 1, 1, d, t)
    k = (k.float() * torch.linspace(0, 12, S, device="cuda").view(1, S, 1, 1)).to(t)
    check(q, k, v, do)
    check(q, k.flip(1), v, do, 300, 7)


def test_strides():
    """Packed projections, sequence-first orders, spread-out gradients: read in place."""
    t, B, S, Hq, Hkv, d = torch.bfloat16, 2, 150, 4, 2, 64
    packed = random(B, S, (Hq + 2 * Hkv), d, dtype=t, seed=1)
    q, k, v = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:]
    first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    heads = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    do = random(B, S, Hq, d, dtype=t, seed=2)
    want = check(q, k, v, do, 70, 4)
    for x in (first, heads, [y.contiguous() for y in (q, k, v)]):
        got = check(*x, do, 70, 4)
        for a, b in zip((got[0], *got[2]), (want[0], *want[2])):
            assert torch.equal(a, b)
    spread = [x[:1].expand(B, S, -1, d) for x in (q, k, v)]
    got = check(*spread, do, 70, 4)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][0])
    one = [x[:, :, :1].expand(B, S, 2, d) for x in (q, k, v)]
    check(*one, do[:, :, :2], 70, 4)
    out = torch.full((B, S, Hq + 1, d), 7.0, dtype=t, device="cuda")
    o, _ = attention.forward(q, k, v, 70, 4, out=out[:, :, 1:])
    assert torch.equal(o, want[0]) and bool((out[:, :, 0] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v", "q", "do"])
@pytest.mark.parametrize("at", [0, 5, 60, 130, 299])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_seen_has_no_part(where, bad, at, d):
    """One value of one token that is no number: rows that do not see it, or that it does not see, are as before."""
    S, window, sinks = 300, 90, 3
    x = dict(zip(("q", "k", "v", "do"), tensors(1, S, S, 2, 1, d, torch.bfloat16)))
    r = Attention(*(f64(x[n])[0] for n in ("q", "k", "v")), window, sinks, d ** -0.5, u(torch.bfloat16))
    want, bound = r.backward(f64(x["do"])[0], r.o_bound)
    x[where][0, at, 0, 7] = bad
    o, lse = attention.forward(x["q"], x["k"], x["v"], window, sinks)
    dq, dk, dv = attention.backward(x["do"], x["q"], x["k"], x["v"], o, lse, window, sinks)
    sees = r.sees
    if where in ("k", "v"):
        touched = sees[:, at]                                   # queries
        keys = sees[touched].any(0)                             # keys that share a query with it
    else:
        touched, keys = np.arange(S) == at, sees[at]
    every = np.ones(S, dtype=bool)
    for got, w, e, rows in ((o, r.o, r.o_bound, every if where == "do" else ~touched),
                            (dq, want["dq"], bound["dq"], ~touched), (dk, want["dk"], bound["dk"], ~keys),
                            (dv, want["dv"], bound["dv"], ~keys)):
        close(got[0][torch.from_numpy(rows).cuda()], w[rows], e[rows])
    if bad != bad and where != "do":
        heads = slice(None) if where in ("k", "v") else 0
        assert bool(torch.isnan(o[0][torch.from_numpy(touched).cuda()][:, heads].float()).any(-1).all())


def test_a_whole_tensor_of_nan():
    q, k, v, do = tensors(1, 260, 260, 2, 1, 64, torch.bfloat16)
    o, lse = attention.forward(torch.full_like(q, float("nan")), k, v, 100, 2)
    assert bool(torch.isnan(o).all())
    for g in attention.backward(do, torch.full_like(q, float("nan")), k, v, o, lse, 100, 2):
        assert bool(torch.isnan(g).all())


def test_results_repeat():
    q, k, v, do = tensors(2, 700, 700, 4, 2, 128, torch.bfloat16)
    o, lse = attention.forward(q, k, v, 300, 4)
    g = attention.backward(do, q, k, v, o, lse, 300, 4)
    for _ in range(3):
        o2, lse2 = attention.forward(q, k, v, 300, 4)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(g, attention.backward(do, q, k, v, o, lse, 300, 4)))


def test_nothing_is_written_outside():
    t, S, H, d = torch.bfloat16, 133, 3, 40
    q, k, v, do = tensors(2, S, S, H, H, d, t)
    store = torch.full((2, S + 2, H + 1, d + 8), 7.0, dtype=t, device="cuda")
    out = store[:, 1:S + 1, :H, :d]
    o, _ = attention.forward(q, k, v, 50, 1, out=out)
    assert o is out and torch.equal(out, attention.forward(q, k, v, 50, 1)[0])
    store[:, 1:S + 1, :H, :d] = 7.0
    assert bool((store == 7).all())


def test_sizes_of_zero():
    t = torch.bfloat16
    for B, Sq, Sk, Hq, Hkv in [(0, 5, 5, 2, 1), (2, 0, 5, 2, 1), (2, 5, 0, 2, 1), (2, 0, 0, 2, 1), (2, 5, 5, 0, 1), (2, 5, 5, 0, 0)]:
        q, k, v, do = tensors(B, Sq, Sk, Hq, Hkv, 64, t)
        o, lse = attention.forward(q, k, v, 3, 1)
        assert o.shape == q.shape and bool((o == 0).all() if Sk == 0 else True) and bool(torch.isneginf(lse).all() if Sk == 0 else True)
        dq, dk, dv = attention.backward(do, q, k, v, o, lse, 3, 1)
        assert dq.shape == q.shape and dk.shape == k.shape and dv.shape == v.shape
        if Sk == 0:
            assert bool((dq == 0).all())
        if Sq == 0 or Hq == 0:
            assert bool((dk == 0).all()) and bool((dv == 0).all())


def test_autograd():
    q, k, v, do = tensors(2, 200, 200, 4, 2, 64, torch.bfloat16)
    rest = torch.empty_like(q, dtype=torch.int8)
    o, lse = attention.forward(q, k, v, 64, 4, rest=rest)
    want = attention.backward(do, q, k, v, o, lse, 64, 4, rest=rest)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    got = autograd.attention(*leaves, window=64, sinks=4)
    got.backward(do)
    assert torch.equal(got, o)
    for a, b in zip(leaves, want):
        assert torch.equal(a.grad, b)
    for need in range(1, 8):
        leaves = [x.clone().requires_grad_(bool(need >> i & 1)) for i, x in enumerate((q, k, v))]
        autograd.attention(*leaves, window=64, sinks=4).backward(do)
        for i, (a, b) in enumerate(zip(leaves, want)):
            assert torch.equal(a.grad, b) if need >> i & 1 else a.grad is None
    one = [x.clone().requires_grad_() for x in (q, k, v)]
    autograd.attention(*one, window=64, sinks=4).sum().backward()            # a gradient spread from one value
    ones = attention.backward(torch.ones_like(do), q, k, v, o, lse, 64, 4, rest=rest)
    assert all(torch.equal(a.grad, b) for a, b in zip(one, ones))


def test_gradient_against_differences():
    """Of the 64-bit form (step 2^-12: off by its square times a third derivative of order one)."""
    S, d, step, window, sinks = 40, 16, 2.0 ** -12, 11, 2
    q, k, v, do = tensors(1, S, S, 2, 1, d, torch.float16)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    autograd.attention(*leaves, window=window, sinks=sinks).backward(do)
    ways = [np.random.default_rng(s).standard_normal(x.shape[1:]) for s, x in enumerate((q, k, v))]

    def value(s):
        a = Attention(*(f64(x)[0] + s * w for x, w in zip((q, k, v), ways)), window, sinks, d ** -0.5, 0)
        return (a.o * f64(do)[0]).sum()

    want = (value(step) - value(-step)) / (2 * step)
    a = Attention(*(f64(x)[0] for x in (q, k, v)), window, sinks, d ** -0.5, u(torch.float16))
    bounds = a.backward(f64(do)[0], a.o_bound)[1]
    got = sum((f64(x.grad)[0] * w).sum() for x, w in zip(leaves, ways))
    room = sum((bounds[n] * np.abs(w)).sum() for n, w in zip(("dq", "dk", "dv"), ways))
    size = sum((np.abs(f64(x.grad)[0]) * np.abs(w)).sum() for x, w in zip(leaves, ways))
    assert abs(got - want) <= room + 2.0 ** -18 * size


# ---- one token over a cache ----------------------------------------------------------

def check_decode(q, k, v, lengths, window=None, sinks=0, scale=None):
    t, d = q.dtype, q.shape[2]
    o = attention.decode(q, k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"), window, sinks, scale)
    assert o.shape == q.shape and o.dtype == t
    for b, n in enumerate(lengths):
        n = max(0, min(n, k.shape[1]))
        if n == 0:
            assert bool((o[b] == 0).all())
            continue
        r = Attention(f64(q[b])[None], f64(k[b, :n]), f64(v[b, :n]), window, sinks, d ** -0.5 if scale is None else scale, u(t))
        close(o[b], r.o[0], r.o_bound[0])
    return o


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (4, 2), (8, 2), (3, 1), (16, 1), (17, 1), (40, 2)])
@pytest.mark.parametrize("d", [64, 128, 8, 40, 80, 120])
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 4)])
def test_decode(Hq, Hkv, d, window, sinks, dtype):
    t = DTYPES[dtype]
    lengths = [0, 1, 2, 31, 64, 65, 300, 513, 700, -3, 900]
    B, cap = len(lengths), 700
    q, k, v = (random(B, *s, dtype=t, seed=i) for i, s in enumerate(((Hq, d), (cap, Hkv, d), (cap, Hkv, d))))
    check_decode(q, k, v, lengths, window, sinks)


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (1, 1), (64, 64), (5000, 3), (700, 150), (1, 5000), (4096, 4)])
@pytest.mark.parametrize("length", [1, 4097, 9000])
def test_decode_long(window, sinks, length):
    cap = 9001
    q, k, v = (random(1, *s, dtype=torch.bfloat16, seed=i) for i, s in enumerate(((8, 64), (cap, 2, 64), (cap, 2, 64))))
    check_decode(q, k, v, [length], window, sinks)


def test_decode_reads_nothing_else():
    """NaN in every place that the token does not see."""
    lengths, window, sinks, cap = [1, 50, 400, 777, 1000], 130, 5, 1000
    q, k, v = (random(5, *s, dtype=torch.bfloat16, seed=i) for i, s in enumerate(((4, 128), (cap, 2, 128), (cap, 2, 128))))
    want = check_decode(q, k, v, lengths, window, sinks)
    for b, n in enumerate(lengths):
        for t in (k, v):
            t[b, n:] = float("nan")
            t[b, min(sinks, max(0, n - window)):max(0, n - window)] = float("inf")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    assert torch.equal(attention.decode(q, k, v, n, window, sinks), want)


def test_decode_strides_and_forward():
    """A cache in any order; and a piece of one query is the same function."""
    cap, Hq, Hkv, d = 333, 4, 2, 64
    q, k, v = (random(3, *s, dtype=torch.float16, seed=i) for i, s in enumerate(((Hq, d), (cap, Hkv, d), (cap, Hkv, d))))
    lengths = [333, 100, 7]
    want = check_decode(q, k, v, lengths, 90, 2)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k2, v2 = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    assert torch.equal(attention.decode(q, k2, v2, n, 90, 2), want)
    out = torch.full((3, Hq + 1, d), 7.0, dtype=torch.float16, device="cuda")
    assert torch.equal(attention.decode(q, k, v, n, 90, 2, out=out[:, 1:]), want) and bool((out[:, 0] == 7).all())
    whole = attention.forward(q[:1, None], k[:1], v[:1], 90, 2)[0]
    r = Attention(f64(q[:1]), f64(k[0]), f64(v[0]), 90, 2, d ** -0.5, u(torch.float16))
    close(whole[0], r.o, r.o_bound)


def test_decode_captured():
    """Lengths are read when the kernel runs: a replay follows them."""
    cap = 600
    q, k, v = (random(2, *s, dtype=torch.bfloat16, seed=i) for i, s in enumerate(((4, 64), (cap, 2, 64), (cap, 2, 64))))
    n = torch.tensor([5, 600], dtype=torch.int32, device="cuda")
    attention.decode(q, k, v, n, 100, 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = attention.decode(q, k, v, n, 100, 4)
    for lengths in ([5, 600], [0, 1], [600, 37]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, attention.decode(q, k, v, n, 100, 4))


def test_step_captured_and_on_another_stream():
    q, k, v, do = tensors(1, 300, 300, 2, 1, 64, torch.bfloat16)
    o, lse = attention.forward(q, k, v, 100, 4)
    want = (o, *attention.backward(do, q, k, v, o, lse, 100, 4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = attention.forward(q, k, v, 100, 4)
        got = (o2, *attention.backward(do, q, k, v, o2, lse2, 100, 4))
    for _ in range(2):
        for g in got:
            g.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3, lse3 = attention.forward(q, k, v, 100, 4)
        got = (o3, *attention.backward(do, q, k, v, o3, lse3, 100, 4))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("scale,size", [(1000.0, 0.03), (30000.0, 0.005), (1e-30, 1.0), (-1e-12, 1.0)])
def test_scales_far_from_one(scale, size, dtype):
    """Scores of a few units under a large scale: lse / scale is small; and under a tiny one, large."""
    q, k, v, do = tensors(1, 190, 200, 2, 1, 64, DTYPES[dtype])
    check(q * size, k * size, v, do, 100, 2, scale)


def test_gradients_past_fp16():
    """dS and D beyond what fp16 holds, the gradients within it."""
    q, k, v, do = tensors(1, 200, 200, 2, 1, 64, torch.float16)
    o, lse = attention.forward(q * 0.02, k * 0.02, v * 40)
    got = attention.backward(do * 400, q * 0.02, k * 0.02, v * 40, o, lse)
    r = Attention(*(f64(x)[0] for x in (q * 0.02, k * 0.02, v * 40)), None, 0, 0.125, u(torch.float16))
    want, bound = r.backward(f64(do * 400)[0], r.o_bound)
    assert np.abs((f64(do * 400)[0] * r.o).sum(-1)).max() > 65504
    for name, g in zip(("dq", "dk"), got):
        close(g[0], want[name], bound[name])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("Sq,Sk,d,window,sinks", [(300, 300, 64, 4, 0), (300, 300, 128, 2, 1), (130, 400, 40, 17, 3),
                                                  (400, 150, 72, None, 0), (1, 1, 8, None, 0)])
def test_what_the_rounding_lost(Sq, Sk, d, window, sinks, dtype):
    """o and `rest` are o with 8 bits more; D, and with it dq and dk, are of both."""
    t = DTYPES[dtype]
    q, k, v, do = tensors(2, Sq, Sk, 4, 2, d, t)
    rest = torch.full(q.shape, 77, dtype=torch.int8, device="cuda")
    o, lse = attention.forward(q, k, v, window, sinks, rest=rest)
    assert torch.equal(o, attention.forward(q, k, v, window, sinks)[0])
    packed = torch.full((2, Sq, 5, d), 77, dtype=torch.int8, device="cuda")
    attention.forward(q, k, v, window, sinks, rest=packed[:, :, 1:])
    assert torch.equal(packed[:, :, 1:], rest) and bool((packed[:, :, 0] == 77).all())
    grads = attention.backward(do, q, k, v, o, lse, window, sinks, rest=rest)
    assert all(torch.equal(a, b) for a, b in zip(grads, attention.backward(do, q, k, v, o, lse, window, sinks, rest=packed[:, :, 1:])))
    # o's bits as a float32, and 256ths of its last place
    both = (o.float().view(torch.int32) + rest.int() * (256 if t == torch.bfloat16 else 32)).view(torch.float32)
    for b in range(2):
        r = Attention(f64(q[b]), f64(k[b]), f64(v[b]), window, sinks, d ** -0.5, u(t))
        # o's own rounding is replaced by half a 256th of the last place; the largest loss, half of it, is one
        # 256th too far; subnormals of fp16 (TINY in o_bound) stay
        less = r.o_bound - u(t) * np.abs(r.o) + u(t) / 64 * (np.abs(r.o) + r.o_bound)
        assert (np.abs(f64(both[b]) - r.o) <= less).all()
        want, bound = r.backward(f64(do[b]), less)
        for name, g in zip(("dq", "dk", "dv"), grads):
            close(g[b], want[name], bound[name])


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_what_the_rounding_lost_of_spread_tensors(dtype):
    """Rows from the definition: keys that are one token's, which TMA cannot address; and a NaN that some do not see."""
    t, S, d = DTYPES[dtype], 150, 64
    q, k, v, do = tensors(1, S, S, 2, 1, d, t)
    r = Attention(f64(q[0]), f64(k[:, :1].expand(1, S, 1, d)[0]), f64(v[0]), 40, 2, d ** -0.5, u(t))
    rest = torch.full(q.shape, 77, dtype=torch.int8, device="cuda")
    o, _ = attention.forward(q, k[:, :1].expand(1, S, 1, d), v, 40, 2, rest=rest)
    def both(rows):
        unit = 256 if t == torch.bfloat16 else 32
        return (o.float().view(torch.int32) + rest.int() * unit).view(torch.float32)[0, rows]
    less = r.o_bound - u(t) * np.abs(r.o) + u(t) / 64 * (np.abs(r.o) + r.o_bound)
    assert (np.abs(f64(both(slice(None))) - r.o) <= less).all()
    r = Attention(f64(q[0]), f64(k[0]), f64(v[0]), 40, 2, d ** -0.5, u(t))
    less = r.o_bound - u(t) * np.abs(r.o) + u(t) / 64 * (np.abs(r.o) + r.o_bound)
    v[0, 70] = float("nan")
    o, _ = attention.forward(q, k, v, 40, 2, rest=rest)
    for rows in (slice(0, 70), slice(110, S)):
        assert (np.abs(f64(both(rows)) - r.o[rows]) <= less[rows]).all()


def test_refusals_of_rest():
    q, k, v, _ = tensors(1, 20, 20, 2, 1, 64, torch.bfloat16)
    whole = torch.zeros(1, 20, 2, 72, dtype=torch.int8, device="cuda")
    for rest in (torch.zeros_like(q), whole[..., :56], whole[..., 4:68], whole.cpu()[..., :64],
                 torch.zeros(1, 20, 2, 68, dtype=torch.int8, device="cuda")[..., :64], 3):
        with pytest.raises(ValueError, match="rest"):
            attention.forward(q, k, v, rest=rest)
    attention.forward(q, k, v, rest=whole[..., 8:])


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 62, 2 ** 62), (50, 2 ** 31 - 1)])
def test_masks_past_every_length(window, sinks):
    q, k, v, do = tensors(1, 150, 200, 2, 1, 64, torch.bfloat16)
    o, lse, g = check(q, k, v, do, window, sinks)
    want = attention.forward(q, k, v)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    lengths = torch.tensor([200], dtype=torch.int32, device="cuda")
    assert torch.equal(attention.decode(q[:, -1], k, v, lengths, window, sinks), attention.decode(q[:, -1], k, v, lengths))


@pytest.mark.parametrize("where", ["k", "v", "q", "do"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_one_token_of_nan_in_a_long_sequence(where, dtype):
    """Rows that do not see it keep their values, also in later rounds of a CTA."""
    S, H, d, at = 2000, 40, 64, 1000
    x = dict(zip(("q", "k", "v", "do"), tensors(1, S, S, H, H, d, DTYPES[dtype])))
    o0, lse0 = attention.forward(x["q"], x["k"], x["v"])
    g0 = attention.backward(x["do"], x["q"], x["k"], x["v"], o0, lse0)
    x[where] = x[where].clone()
    x[where][:, at] = float("nan")
    o, lse = attention.forward(x["q"], x["k"], x["v"])
    dq, dk, dv = attention.backward(x["do"], x["q"], x["k"], x["v"], o, lse)
    rows = torch.arange(S, device="cuda")
    seers = rows >= at if where in ("k", "v") else rows == at            # queries
    seen = rows <= (S - 1 if where in ("k", "v") else at)                 # keys of those
    some = torch.zeros_like(rows, dtype=torch.bool)
    room = 64 * u(DTYPES[dtype])          # a row from the definition has P and dS in 32 bits
    for got, want, lost in ((o, o0, some if where == "do" else seers), (dq, g0[0], seers),
                            (dk, g0[1], seen), (dv, g0[2], some if where == "v" else seen)):
        assert bool(torch.isnan(got[0][lost]).any(-1).all())
        a, b = got[0][~lost].double(), want[0][~lost].double()
        assert bool(((a - b).abs() <= room * b.abs().amax(-1, keepdim=True)).all())


def test_zz_no_wait_ran_out():
    assert basp.basp_attention_timeouts() == 0


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("offset", [1, 3, 4, 8])
def test_gradients_of_a_piece_of_a_buffer(offset, dtype):
    """A contiguous gradient that begins anywhere, as the backward of torch.cat hands it on."""
    q, k, v, _ = tensors(1, 37, 37, 2, 1, 64, DTYPES[dtype])
    grads = []
    for before in (offset, 0):
        leaves = [x.clone().requires_grad_() for x in (q, k, v)]
        o = autograd.attention(*leaves, window=20, sinks=1)
        flat = torch.cat([torch.zeros(before, dtype=q.dtype, device="cuda"), o.reshape(-1)])
        do = random(o.numel(), dtype=q.dtype, seed=5)
        flat.backward(torch.cat([torch.zeros(before, dtype=q.dtype, device="cuda"), do]))
        grads.append([x.grad for x in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*grads))


@pytest.mark.parametrize("path", ["tiles", "rows", "again"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_scores_of_minus_infinity(path, dtype):
    """The first key's, alone among the sinks: it weighs nothing, in the tiles, in the form for
    tensors that TMA cannot address, and in rows that are computed again beside a NaN."""
    t, S, d, window = DTYPES[dtype], 150, 64, 40
    q, k, v, _ = tensors(1, S, S, 2, 1, d, t)
    if path == "rows":
        q = q[:, :1].clone().expand(1, S, 2, d)
    q[..., 7] = 1.0
    k[0, 0, 0, 7] = float("-inf")
    rows = np.arange(1, S)
    if path == "again":
        v[0, 100] = float("nan")
        rows = rows[(rows < 100) | (rows >= 100 + window)]
    o, lse = attention.forward(q, k, v, window, 1)
    # without the first key; rows that see the NaN are left out
    r = Attention(f64(q[0, 1:]), f64(k[0, 1:]), f64(v[0, 1:].nan_to_num()), window, 0, d ** -0.5, u(t))
    close(o[0][torch.from_numpy(rows).cuda()], r.o[rows - 1], r.o_bound[rows - 1])
    close(lse[0, :, 1:], r.lse, r.lse_bound)
    assert bool(torch.isnan(o[0, 0]).all()) and bool(torch.isneginf(lse[0, :, 0]).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["small", "smaller", "subnormal", "rows", "tiles", "large"])
@pytest.mark.parametrize("S,Hq,Hkv,window,sinks", [(700, 2, 1, None, 0), (700, 4, 2, 130, 5), (2500, 1, 1, None, 0), (2500, 2, 1, 100, 300)])
def test_small_gradients_in_fp16(S, Hq, Hkv, window, sinks, kind, d):
    """dS far below what fp16 is exact to: it is rounded as a power of two times it, 1 to 2 over
    the largest |do| of a query (dq), or of all queries of the heads (dk, at least), and P of dv
    as 2^10 times it.  So that dq and dk are not subnormal themselves, q and k are 2^-8 as large
    and the scale of their products 2^16: the same scores, and gradients 2^8 as large."""
    t = torch.float16
    q, k, v, do = tensors(1, S, S, Hq, Hkv, d, t)
    n = torch.arange(S, device="cuda").view(1, S, 1, 1)
    size = {"small": 2.0 ** -10, "smaller": 2.0 ** -13, "subnormal": 2.0 ** -19, "rows": torch.exp2(-(n * 7 % 20).float()),
            "tiles": torch.exp2(-(n // 128 % 3 * 6).float()), "large": 2.0 ** 10}[kind]
    do = (do.float() * size).to(t)
    scale = d ** -0.5
    if kind != "large":
        q, k, scale = q * 2.0 ** -8, k * 2.0 ** -8, scale * 2.0 ** 16
    o, lse = attention.forward(q, k, v, window, sinks, scale)
    got = attention.backward(do, q, k, v, o, lse, window, sinks, scale)
    r = Attention(f64(q[0]), f64(k[0]), f64(v[0]), window, sinks, scale, u(t))
    top = np.abs(f64(do[0])).max(-1).T                                          # [hq, sq]
    want, bound = gradients_in_units(r, f64(do[0]), r.o_bound, 2.0 ** 10, 1 / top, 1 / top.max())
    for name, g in zip(("dq", "dk", "dv"), got):
        close(g[0], want[name], bound[name])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 2.0])
@pytest.mark.parametrize("S,Hq,Hkv,window,sinks", [(300, 2, 1, 2, 0), (2500, 2, 1, 3, 4), (700, 4, 2, 1, 1), (300, 1, 1, None, 0)])
def test_past_fp16(S, Hq, Hkv, window, sinks, size, d):
    """dS past what fp16 holds in units of do, in tiles of keys that CTAs share too; with heads
    of 128 or twice the gradient, D past what its parts hold: such rows are the definition's."""
    t = torch.float16
    q, k, v, do = tensors(1, S, S, Hq, Hkv, d, t)
    v = (v[..., :1].float().sign() * 60000).to(t).expand(1, S, Hkv, d).contiguous()      # one sign a token
    q, k, do = q * 2.0 ** -12, k * 2.0 ** -12, torch.full_like(do, size)
    o, lse = attention.forward(q, k, v, window, sinks)
    got = attention.backward(do, q, k, v, o, lse, window, sinks)
    r = Attention(f64(q[0]), f64(k[0]), f64(v[0]), window, sinks, d ** -0.5, u(t))
    want, bound = r.backward(f64(do)[0], r.o_bound)
    assert max(np.abs(r.p[h] * (f64(do)[0, :, h] @ f64(v)[0, :, h // (Hq // Hkv)].T)).max() for h in range(Hq)) > 2 * 65504 * size
    for name, g in zip(("dq", "dk", "dv"), got):
        close(g[0], want[name], bound[name])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v", "q", "do"])
@pytest.mark.parametrize("at", [0, 60, 130, 299])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_seen_has_no_part_in_fp16(where, bad, at, d):
    """As above; and rows that do see a NaN are NaN by the tiles' answer."""
    S, window, sinks = 300, 90, 3
    x = dict(zip(("q", "k", "v", "do"), tensors(1, S, S, 2, 1, d, torch.float16)))
    r = Attention(*(f64(x[n])[0] for n in ("q", "k", "v")), window, sinks, d ** -0.5, u(torch.float16))
    want, bound = r.backward(f64(x["do"])[0], r.o_bound)
    x[where][0, at, 0, 7] = bad
    o, lse = attention.forward(x["q"], x["k"], x["v"], window, sinks)
    grads = attention.backward(x["do"], x["q"], x["k"], x["v"], o, lse, window, sinks)
    sees = r.sees
    touched = sees[:, at] if where in ("k", "v") else np.arange(S) == at
    keys = sees[touched].any(0)
    for name, g, rows in zip(("dq", "dk", "dv"), grads, (touched, keys, keys)):
        close(g[0][torch.from_numpy(~rows).cuda()], want[name][~rows], bound[name][~rows])
    if bad != bad:
        heads = slice(None) if where in ("k", "v") else 0
        assert bool(torch.isnan(grads[0][0][torch.from_numpy(touched).cuda()][:, heads].float()).any(-1).all())
        assert bool(torch.isnan(grads[1][0][torch.from_numpy(keys).cuda()].float()).any(-1).all())


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_one_overflow_costs_little(dtype):
    """An infinity in the last query's gradient makes every key's row no number: that is the
    tiles' answer, and no row is walked again for it.  (Walked, it was some hundred times as long.)"""
    S, H, d = 8192, 8, 64
    q, k, v, do = tensors(1, S, S, H, H, d, DTYPES[dtype])
    o, lse = attention.forward(q, k, v)

    def best():
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            got = attention.backward(do, q, k, v, o, lse)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times), got

    plain, _ = best()
    do[0, S - 1, :, 3] = float("inf")
    bad, (dq, dk, dv) = best()
    assert bool(torch.isfinite(dq[0, :S - 1]).all()) and not bool(torch.isfinite(dk).any()) and not bool(torch.isfinite(dv[..., 3]).any())
    assert bad <= 40 * plain


@pytest.mark.parametrize("S,Hq,Hkv,d,window,sinks", [(700, 4, 2, 128, 300, 4), (2500, 2, 1, 64, 100, 300), (130, 6, 2, 96, None, 0)])
def test_results_repeat_in_fp16(S, Hq, Hkv, d, window, sinks):
    """Units and bounds are made anew by each call, in a graph and on another stream too, whatever
    its workspace held before."""
    x = tensors(2, S, S, Hq, Hkv, d, torch.float16)
    y = [t * 2.0 ** -8 for t in x]
    o, lse = attention.forward(*x[:3], window, sinks)
    want = attention.backward(x[3], *x[:3], o, lse, window, sinks)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attention.backward(x[3], *x[:3], o, lse, window, sinks)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        attention.backward(y[3] * 2.0 ** -9, *x[:3], o, lse, window, sinks)          # another unit, the same memory
        for g in got:
            g.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            beside = attention.backward(x[3], *x[:3], o, lse, window, sinks)
        again = attention.backward(x[3], *x[:3], o, lse, window, sinks)
        torch.cuda.synchronize()
        for grads in (got, beside, again):
            assert all(torch.equal(a, b) for a, b in zip(grads, want))


def is_shared(Sq, Sk, Hq, Hkv, d, window, sinks, dtype, batch=1):
    """Whether CTAs share a tile of keys: then the workspace holds their parts' sums beside the
    rows' statistics (40 bytes a query of whole tiles) and fp16's units (less than 5, and a number a tile of keys)."""
    desc = basp.basp_attention_desc(batch, Sq, Sk, Hq, Hkv, d, window or 0, sinks, d ** -0.5, basp.DTYPE_CODES[dtype])
    rows, tiles = batch * Hq * (-(-Sq // 128) * 128), batch * Hkv * -(-Sk // 128)
    own = rows * 40 + ((rows * 4 + rows // 32 * 16 + -(-tiles // 4) * 16) if dtype == "fp16" else 0)
    got = basp.basp_attention_backward_workspace(desc)
    assert got >= own
    return got > own


SHARED = [(2300, 2300, 4, 1, 64, 100, 3), (2300, 2300, 5, 1, 128, None, 0), (2000, 2501, 10, 2, 40, 300, 200),
          (1500, 2001, 8, 1, 72, 64, 700), (20000, 20000, 1, 1, 64, 50, 2)]


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("Sq,Sk,Hq,Hkv,d,window,sinks", SHARED[:4])
def test_shared_key_tiles(Sq, Sk, Hq, Hkv, d, window, sinks, dtype):
    t = DTYPES[dtype]
    assert is_shared(Sq, Sk, Hq, Hkv, d, window, sinks, dtype)
    q, k, v, do = tensors(1, Sq, Sk, Hq, Hkv, d, t)
    o, lse, g = check(q, k, v, do, window, sinks)
    assert all(torch.equal(a, b) for a, b in zip(g, attention.backward(do, q, k, v, o, lse, window, sinks)))
    bad = do.clone()
    bad[0, Sq // 2, 0, 3] = float("nan")
    r = Attention(*(f64(x)[0] for x in (q, k, v)), window, sinks, d ** -0.5, u(t))
    want, bound = r.backward(f64(do)[0], r.o_bound)
    rows = ~r.sees[Sq // 2]
    got = attention.backward(bad, q, k, v, o, lse, window, sinks)
    for name, x in zip(("dk", "dv"), got[1:]):
        close(x[0][torch.from_numpy(rows).cuda()], want[name][rows], bound[name][rows])
    assert bool(torch.isnan(got[1][0, :, 0][torch.from_numpy(~rows).cuda()]).all())        # the first query head's key head
    assert bool(torch.isfinite(got[1][0, :, 1:]).all())


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_shared_key_tiles_of_a_long_sequence(dtype):
    """One head: its first keys' dk and dv in 64 bits, from the lse and o that the backward gets."""
    Sq, Sk, Hq, Hkv, d, window, sinks = SHARED[4]
    assert is_shared(Sq, Sk, Hq, Hkv, d, window, sinks, dtype)
    t = DTYPES[dtype]
    q, k, v, do = tensors(1, Sq, Sk, Hq, Hkv, d, t)
    o, lse = attention.forward(q, k, v, window, sinks)
    dq, dk, dv = attention.backward(do, q, k, v, o, lse, window, sinks)
    n, s = 4, d ** -0.5
    qd, kd, vd, dod = (x[0, :, 0].double() for x in (q, k, v, do))
    first = kd[:n]
    p = torch.exp(s * qd @ first.T - lse[0, 0].double()[:, None])
    i, j = torch.arange(Sq, device="cuda")[:, None], torch.arange(n, device="cuda")
    p = p * ((j <= i) & ((j > i - window) | (j < sinks)))
    ds = p * (dod @ vd[:n].T - (dod * o[0, :, 0].double()).sum(1, keepdim=True))
    for got, want, size in ((dv, p.T @ dod, p.T @ dod.abs()), (dk, s * ds.T @ qd, s * ds.abs().T @ qd.abs())):
        room = 4 * u(t) * size + u(t) * want.abs() + 2.0 ** -24
        assert bool(((got[0, :n, 0].double() - want).abs() <= room).all())
    assert bool(torch.isfinite(dq).all())


@pytest.mark.parametrize("size", [1.0, 2.0])
@pytest.mark.parametrize("d", [64, 128])
def test_past_fp16_in_shared_tiles(d, size):
    """As test_past_fp16: the parts of a shared tile say it to the kernel that adds them."""
    t, S, Hq, window, sinks = torch.float16, 1300, 8, 3, 4
    assert is_shared(S, S, Hq, 1, d, window, sinks, "fp16")
    q, k, v, do = tensors(1, S, S, Hq, 1, d, t)
    v = (v[..., :1].float().sign() * 60000).to(t).expand(1, S, 1, d).contiguous()
    q, k, do = q * 2.0 ** -14, k * 2.0 ** -14, torch.full_like(do, size)
    o, lse = attention.forward(q, k, v, window, sinks)
    got = attention.backward(do, q, k, v, o, lse, window, sinks)
    r = Attention(f64(q[0]), f64(k[0]), f64(v[0]), window, sinks, d ** -0.5, u(t))
    want, bound = r.backward(f64(do)[0], r.o_bound)
    for name, g in zip(("dq", "dk", "dv"), got):
        close(g[0], want[name], bound[name])


@pytest.mark.parametrize("kind", ["smaller", "rows", "tiles"])
def test_small_gradients_in_shared_tiles(kind):
    """Each part of a shared tile has a unit of its own."""
    assert is_shared(1500, 1500, 6, 1, 64, None, 0, "fp16")
    test_small_gradients_in_fp16(1500, 6, 1, None, 0, kind, 64)


def test_zzz_no_wait_ran_out_either():
    assert basp.basp_attention_timeouts() == 0
