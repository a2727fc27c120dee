"""Attention, layer norm and the optimiser's step on tensors of more than 2^31 elements,
and calls on two streams at a time."""
import numpy as np
import pytest
import torch

import sequence_re_layout_gb300 as basp
from layer_reference import Attention
from sequence_re_layout_gb300 import attention, fp8, optim
from test_gpu_attention import _built, close, f64, random, u         # noqa: F401

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def room():
    """These take tens of GB, which no other test's cache should hold."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def long_cache(S, H, d, ends):
    """[1, S, H, d] of NaN, but for the first 5 tokens and the last `ends`."""
    t = torch.full((1, S, H, d), float("nan"), dtype=BF16, device="cuda")
    t[:, :5] = random(1, 5, H, d, dtype=BF16, seed=S + 1)
    t[:, S - ends:] = random(1, ends, H, d, dtype=BF16, seed=S + 2)
    return t, torch.cat([t[:, :5], t[:, S - ends:]], 1)


def test_a_long_cache():
    """What is behind 2^31 elements of keys is found there; nothing between sinks and window is read."""
    S, H, d, Sq, window, ends = (1 << 21) + 7777, 8, 128, 200, 300, 600
    (k, few_k), (v, few_v) = long_cache(S, H, d, ends), long_cache(S, H, d, ends)
    assert k.numel() > 1 << 31
    q, do = random(1, Sq, H, d, dtype=BF16, seed=3), random(1, Sq, H, d, dtype=BF16, seed=4)
    r = Attention(f64(q[0]), f64(few_k[0]), f64(few_v[0]), window, 5, d ** -0.5, u(BF16))
    want, bound = r.backward(f64(do[0]), r.o_bound)
    o, lse = attention.forward(q, k, v, window, 5)
    close(o[0], r.o, r.o_bound)
    dq, dk, dv = attention.backward(do, q, k, v, o, lse, window, 5)
    close(dq[0], want["dq"], bound["dq"])
    for name, g in (("dk", dk), ("dv", dv)):
        close(torch.cat([g[0, :5], g[0, S - ends:]]), want[name], bound[name])
        assert not bool(g[0, 5:S - ends].any())
    lengths = torch.tensor([S], dtype=torch.int32, device="cuda")
    one = attention.decode(q[:, -1], k, v, lengths, window, 5)
    few = attention.decode(q[:, -1], few_k, few_v, torch.full_like(lengths, ends + 5), window, 5)
    assert torch.equal(one, few)


def test_a_batch_of_long_caches():
    B, S, H, d = 3, 1 << 20, 8, 128
    k, v = (torch.zeros(B, S, H, d, dtype=BF16, device="cuda") for _ in range(2))
    k[2, :400], v[2, :400] = random(400, H, d, dtype=BF16, seed=1), random(400, H, d, dtype=BF16, seed=2)
    v[1, -1] = 1.0
    q = random(B, H, d, dtype=BF16, seed=3)
    lengths = torch.tensor([0, S, 400], dtype=torch.int32, device="cuda")
    got = attention.decode(q, k, v, lengths)
    assert not bool(got[0].any()) and bool(((got[1].double() * S - 1).abs() <= 0.01).all())      # all scores 0
    r = Attention(f64(q[2:]), f64(k[2, :400]), f64(v[2, :400]), None, 0, d ** -0.5, u(BF16))
    close(got[2:], r.o, r.o_bound)


@pytest.mark.parametrize("quantized", [False, True])
def test_layernorm_of_far_rows(quantized):
    rows, cols, stride = 300, 520, 1 << 23
    store = torch.empty(rows, stride, dtype=BF16, device="cuda")
    x = store[:, 8:8 + cols]
    x.copy_(random(rows, cols, dtype=BF16, seed=1))
    w, b = random(cols, dtype=BF16, seed=2), random(cols, dtype=BF16, seed=3)
    far, near = fp8.layernorm(x, w, b, quantized=quantized), fp8.layernorm(x.contiguous(), w, b, quantized=quantized)
    for a, c in zip(far[:1] + far[2:], near[:1] + near[2:]):
        a, c = (y.data.view(torch.uint8) if isinstance(y, fp8.Quantized) else y for y in (a, c))
        assert torch.equal(a, c)
    dy = store[:, 4096:4096 + cols]
    dy.copy_(random(rows, cols, dtype=BF16, seed=4))
    for a, c in zip(fp8.layernorm_backward(dy, x, far[2], far[3], w, dh=dy),
                    fp8.layernorm_backward(dy.contiguous(), x.contiguous(), far[2], far[3], w, dh=dy.contiguous())):
        assert torch.equal(a, c)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_large_tensor(bits):
    n, tail = (1 << 31) + 128 * 3, 1000
    p, g = torch.ones(n, dtype=BF16, device="cuda"), torch.empty(n, dtype=BF16, device="cuda")
    g.fill_(0.5)
    g[-tail:] = random(tail, dtype=BF16, seed=1)
    if bits == 32:
        m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    else:
        def zero():
            return fp8.Quantized(torch.zeros(1, n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                                 torch.zeros(1, n // 128, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu))
        m, v = zero(), zero()
    optim.adamw([p], [g], [m], [v], 1, lr=0.25, weight_decay=0.0)
    few = [torch.ones(tail, dtype=BF16, device="cuda"), g[-tail:].clone(), torch.zeros(tail, device="cuda"),
           torch.zeros(tail, device="cuda")]
    optim.adamw(*([x] for x in few), 1, lr=0.25, weight_decay=0.0)
    assert torch.equal(p[-tail:], few[0])
    assert bool((p[:-tail] == 0.75).all())
    if bits == 32:
        assert torch.equal(m[-tail:], few[2]) and torch.equal(v[-tail:], few[3])
    else:
        for s, want in ((m, few[2]), (v, few[3].sqrt())):
            got = s.data[0, -896:].float() * torch.exp2(s.scales[0, -7:].view(torch.uint8).float() - 127).repeat_interleave(128)
            # one step of e4m3: 2^-3 of the value, or 2^-9 of the scale, which is at most the largest / 224
            assert bool(((got - want[-896:]).abs() <= want[-896:].abs() / 8 + want.abs().max() / 224 / 512).all())


def test_two_streams_at_a_time():
    """Calls of every kind on two streams keep apart: the results are those of one after the other."""
    S, H, d = 1500, 8, 64
    def inputs(i):
        t = [random(2, S, H, d, dtype=BF16, seed=10 * i + j) for j in range(4)]
        return t, random(4000, 1024, dtype=BF16, seed=10 * i + 5), torch.tensor([S, 700], dtype=torch.int32, device="cuda")

    def work(x):
        (q, k, v, do), a, lengths = x
        o, lse = attention.forward(q, k, v, 200, 4)
        grads = attention.backward(do, q, k, v, o, lse, 200, 4)
        w = a[0].contiguous()
        y, _, mean, rstd = fp8.layernorm(a, w, quantized=False)
        back = fp8.layernorm_backward(y, a, mean, rstd, w)
        p, m, s = a.clone(), torch.zeros(a.shape, device="cuda"), torch.zeros(a.shape, device="cuda")
        optim.adamw([p], [back[0]], [m], [s], 1)
        return [o, lse, *grads, y, mean, rstd, *back, p, m, s, attention.decode(q[:, 0].contiguous(), k, v, lengths)]

    x = [inputs(0), inputs(1)]
    want = [work(i) for i in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for i, s in zip(x, streams):
            with torch.cuda.stream(s):
                got.append(work(i))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(c, e) for c, e in zip(a, b))
    assert np.isfinite(f64(want[0][0])).all()


def test_two_graphs_at_a_time():
    """Two captured calls of each kind, replayed on two streams at once, share no workspace."""
    S, H, d = 1200, 4, 128
    x = [[random(2, S, H, d, dtype=BF16, seed=20 * i + j) for j in range(4)] for i in range(2)]
    lengths = torch.tensor([S, 321], dtype=torch.int32, device="cuda")

    def work(q, k, v, do):
        rest = torch.empty(q.shape, dtype=torch.int8, device="cuda")
        o, lse = attention.forward(q, k, v, None, 0, rest=rest)
        a, w = q.view(-1, H * d), k.view(-1, H * d)[0]
        y, _, mean, rstd = fp8.layernorm(a, w, quantized=False)
        return [o, lse, rest, *attention.backward(do, q, k, v, o, lse, rest=rest),
                attention.decode(q[:, -1], k, v, lengths), *fp8.layernorm_backward(y, a, mean, rstd, w)]

    want = [work(*i) for i in x]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, i in zip(graphs, x):
        with torch.cuda.graph(g):
            got.append(work(*i))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(c, e) for c, e in zip(a, b))


def test_zz_no_wait_ran_out():
    assert basp.basp_attention_timeouts() == 0
