"""A whole training step of the layer in examples/attention_layer.py: norm, 8-bit
projections, re-layout, attention with a window and sinks, and AdamW; against the same
step in 64 bits, captured in a graph, and with everything in one run."""
import os
import subprocess
import sys

import pytest
import torch

import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import attention, autograd, optim
from test_gpu_projections import ROOT, _built, example            # noqa: F401

pytestmark = pytest.mark.gpu


def plain_layer(layer, x, residual, B, S, window, sinks):
    """The layer on full-precision leaves, in 64 bits on sequences in order."""
    i = layer.layout.info
    leaves = [p.detach().double().requires_grad_() for p in layer.parameters()]
    nw, nb, wqkv, bqkv, wo = (dict(zip(dict(layer.named_parameters()), leaves))[n]
                              for n in ("norm", "norm_bias", "wqkv", "bqkv", "wo"))
    h = (x + residual).double()
    y = torch.nn.functional.layer_norm(h, h.shape[-1:], nw, nb, 1e-5)
    qkv = (y @ wqkv.T + bqkv).view(B, S, -1, i["d"])
    q, k, v = (t.transpose(1, 2) for t in qkv.split([i["Hq"], i["Hkv"], i["Hkv"]], dim=2))
    k, v = (t.repeat_interleave(i["Hq"] // i["Hkv"], 1) for t in (k, v))
    p, j = torch.arange(S, device="cuda")[:, None], torch.arange(S, device="cuda")
    mask = (j <= p) & ((j > p - window) | (j < sinks))
    p = torch.softmax((q @ k.transpose(-1, -2) * i["d"] ** -0.5).masked_fill(~mask, float("-inf")), -1)
    return (p @ v).transpose(1, 2).reshape(B, S, -1) @ wo.T, h, leaves


@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("bits", [32, 8])
def test_training_step(K, bits):
    """Operands in 8 bits move a product by 0.09 of itself (tests/test_gpu_projections.py),
    the layer's output by 0.2, its gradients by less than 0.35.  The first step of Adam is
    lr times a sign, wherever the gradient is not near zero: the weights move the same way
    where 64 bits have a gradient of more than its own root mean square."""
    B, S, Hq, Hkv, d, N, window, sinks = 2, 256, 8, 4, 64, 4, 60, 3
    torch.manual_seed(1)
    with basp.Layout(B, S, Hq, Hkv, d, N, K, "bf16") as L:
        layer = example().AttentionLayer(L, Hq * d, norm="layer", window=window, sinks=sinks)
        optimizer = optim.AdamW(layer.parameters(), lr=0.0625, weight_decay=0.0, state_bits=bits)
        bg, per = B // (N // K), S // K
        shards = lambda t: t.view(N // K, bg, K, per, -1).transpose(1, 2).reshape(B * S, -1)     # noqa: E731
        whole = lambda t: t.view(N // K, K, bg, per, -1).transpose(1, 2).reshape(B, S, -1)       # noqa: E731
        x, r, dy = (torch.randn(B, S, Hq * d, device="cuda").bfloat16() for _ in range(3))
        want, want_h, leaves = plain_layer(layer, x, r, B, S, window, sinks)
        want.backward(dy.double())
        before = [p.detach().clone() for p in layer.parameters()]
        out, h = layer(shards(x), shards(r))
        out.backward(shards(dy))
        error = whole(out.detach()).double() - want.detach()
        assert float(error.norm() / want.detach().norm()) <= 0.2 and torch.equal(whole(h), x + r)
        optimizer.step()
        for p, old, leaf in zip(layer.parameters(), before, leaves):
            assert float(torch.nn.functional.cosine_similarity(p.grad.double().flatten(), leaf.grad.flatten(), 0)) >= 0.9
            large = leaf.grad.abs() > leaf.grad.square().mean().sqrt()
            moved = (p.detach().double() - old.double())[large]
            assert float((torch.sign(moved) == -torch.sign(leaf.grad[large])).double().mean()) >= 0.99
            room = 2.0 ** -7 * old.double().abs()[large] + 2.0 ** -12       # p's own type, and the quotient
            assert bool(((moved.abs() - 0.0625).abs() <= room).all())
        layer.freeze()
        with torch.no_grad():
            assert bool(torch.isfinite(layer(shards(x), shards(r))[0]).all())


def test_training_steps_in_a_graph():
    """Forward, backward and optimiser captured together and replayed; eager steps of a
    second layer give the same weights."""
    B, S, Hq, Hkv, d, N, K = 2, 256, 8, 4, 64, 4, 2
    with basp.Layout(B, S, Hq, Hkv, d, N, K, "bf16") as L:
        layers, opts = [], []
        for _ in range(2):
            torch.manual_seed(3)
            layers.append(example().AttentionLayer(L, Hq * d, norm="layer", window=70, sinks=2))
            opts.append(optim.AdamW(layers[-1].parameters(), lr=0.01, state_bits=8, capturable=True))
        x, r, target = (torch.randn(B * S, Hq * d, device="cuda").bfloat16() for _ in range(3))

        def step(layer, opt):
            opt.zero_grad(set_to_none=False)
            out, h = layer(x, r)
            (out + h - target).float().square().mean().backward()
            opt.step()

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                step(layers[0], opts[0])
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(layers[0], opts[0])
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for _ in range(5):
            step(layers[1], opts[1])
        for a, b in zip(layers[0].parameters(), layers[1].parameters()):
            assert torch.equal(a, b)


def test_tokens_one_by_one():
    """A prompt in one piece, then tokens over the cache, are a longer prompt's rows: within
    the roundings of their type (one of P, one of the result: 2^-8 of the values' sizes each)."""
    B, S, n, Hq, Hkv, d, window, sinks = 2, 300, 260, 8, 2, 64, 100, 4
    torch.manual_seed(5)
    q, k, v = (torch.randn(B, S, h, d, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    want = attention.forward(q, k, v, window, sinks)[0]
    cache_k, cache_v = (torch.full((B, S + 20, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache_k[:, :n], cache_v[:, :n] = k[:, :n], v[:, :n]
    prompt = attention.forward(q[:, :n], cache_k[:, :n], cache_v[:, :n], window, sinks)[0]
    assert torch.equal(prompt, want[:, :n])
    tail = attention.forward(q[:, n:], k, v, window, sinks)[0]
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    for t in range(n, S):
        cache_k[:, t], cache_v[:, t] = k[:, t], v[:, t]
        lengths += 1
        got = attention.decode(q[:, t], cache_k, cache_v, lengths, window, sinks)
        for a, b in ((got, want[:, t]), (tail[:, t - n], want[:, t])):
            assert bool(((a.float() - b.float()).abs() <= 4 * 2.0 ** -8 * (v.float().abs().max() / 8 + b.float().abs())).all())


@pytest.mark.parametrize("extra", [["--norm", "layer", "--window", "100", "--sinks", "4", "--state-bits", "8"],
                                   ["--workload", "llama3.2-1b_B2_S8192"]])
def test_example_program(extra):
    """It runs; nothing is asked of the losses but that they are numbers."""
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "attention_layer.py"), "--seq", "512", "--steps", "2",
                        *extra], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    losses = [float(line.split()[-1]) for line in r.stdout.splitlines() if "loss" in line]
    assert len(losses) == 3 and all(x == x and abs(x) < float("inf") for x in losses), r.stdout


def test_zz_no_wait_ran_out():
    assert basp.basp_attention_timeouts() == 0 and basp.basp_matmul_fp8_timeouts() == 0


@pytest.mark.parametrize("dims", [(0,), (1,), (2,), (0, 1), (0, 1, 2, 3)])
def test_spread_gradients(dims):
    """A gradient that is one value, one token's or one head's, spread over the result."""
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, 140, h, 64, generator=g).bfloat16().cuda().requires_grad_() for h in (4, 2, 2))
    shape = [1 if i in dims else n for i, n in enumerate(q.shape)]
    do = torch.randn(shape, generator=g).bfloat16().cuda()
    got = torch.autograd.grad(autograd.attention(q, k, v, 60, 3), (q, k, v), do.expand(q.shape))
    want = torch.autograd.grad(autograd.attention(q, k, v, 60, 3), (q, k, v), do.expand(q.shape).contiguous())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
