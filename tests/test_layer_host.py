"""CPU checks of the C ABIs of include/basp_attention.h, include/basp_optim.h and the
layer norm of include/basp_fp8.h: exported symbols, and refusals, which all happen
before anything reaches a GPU; and of the 64-bit forms that the GPU tests compare with."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import layer_reference as ref
import sequence_re_layout_gb300 as basp
from sequence_re_layout_gb300 import attention, autograd, fp8, optim
from sequence_re_layout_gb300.build import build_library
from test_fp8_host import ALIAS, ALIGN, BF16, FP16, FP32, FP8, GiB, INVALID, LARGE, OK, WORKSPACE, at, q8

DIVIDE = basp.BASP_ERR_DIVISIBILITY
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return basp.load_library()


@pytest.mark.parametrize("header,exports", [("basp_attention.h", basp.ATTENTION_EXPORTS), ("basp_optim.h", basp.OPTIM_EXPORTS)])
def test_every_declared_symbol_is_exported(lib, header, exports):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
    assert set(re.findall(r"\b(basp_\w+)\s*\(", text)) == set(exports)
    for n in exports:
        assert hasattr(lib, n), n


LAYER = dict(dtype=BF16, rows=4, cols=256, x=at(1), xs=256, r=at(2), rs=256, w=at(3), b=at(9), wd=BF16, eps=1e-6,
             h=at(4), hs=256, y=at(5), ys=256, q=None, mean=at(10), rstd=at(6), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), OK), (dict(cols=0, q=q8(7, 4, 0)), OK), (dict(rows=0, x=None, r=None, h=None, rstd=None), OK),
    (dict(dtype=FP8), INVALID), (dict(dtype=9), INVALID), (dict(wd=FP16), INVALID), (dict(rows=-1), INVALID),
    (dict(rows=1 << 31), LARGE), (dict(cols=1 << 31), LARGE), (dict(x=None), INVALID), (dict(w=None), INVALID),
    (dict(y=None, q=None), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(xs=255), INVALID), (dict(x=at(1) + 1), ALIGN), (dict(b=at(9) + 1), ALIGN), (dict(mean=at(10) + 2), ALIGN),
    (dict(y=at(1)), ALIAS), (dict(h=at(1) + 512), ALIAS), (dict(mean=at(6)), ALIAS), (dict(mean=at(9)), ALIAS),
    (dict(q=q8(7, 4, 128)), INVALID), (dict(q=q8(7, 4, 256, 128)), INVALID), (dict(q=q8(7, 4, 256, pitch=264)), ALIGN),
    (dict(q=q8(7, 4, 256, data=at(5))), ALIAS),
])
def test_layernorm_refusals(lib, change, status):
    assert lib.basp_layernorm(*{**LAYER, **change}.values()) == status


LAYER_BACK = dict(dtype=BF16, rows=4, cols=256, dy=at(1), dys=256, h=at(2), hs=256, mean=at(9), rstd=at(3), w=at(4), wd=FP32,
                  dh=at(5), dhs=256, dx=at(6), dxs=256, dw=at(7), db=at(10), ws=at(8), wsb=4 * 2 * 256 * 4, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(cols=0), OK), (dict(rows=0, dw=None, db=None), OK),
    (dict(dtype=FP8), INVALID), (dict(rows=1 << 31), LARGE), (dict(dy=None), INVALID), (dict(h=None), INVALID),
    (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=4 * 2 * 256 * 4 - 1), WORKSPACE), (dict(ws=None, db=None), WORKSPACE),
    (dict(ws=at(8) + 4), ALIGN), (dict(dx=at(2)), ALIAS), (dict(dx=at(1) + 512), ALIAS), (dict(dw=at(10)), ALIAS),
    (dict(db=at(8)), ALIAS), (dict(db=at(10) + 2), ALIGN),
])
def test_layernorm_backward_refusals(lib, change, status):
    assert lib.basp_layernorm_backward(*{**LAYER_BACK, **change}.values()) == status


def test_workspaces():
    assert basp.basp_layernorm_backward_workspace(0, 256) == 0
    assert basp.basp_layernorm_backward_workspace(4, 256) == 4 * 2 * 256 * 4
    assert basp.basp_layernorm_backward_workspace(1 << 20, 256) == basp.basp_layernorm_backward_workspace(1 << 21, 256)


DESC = dict(batch=2, q_len=100, k_len=300, q_heads=6, k_heads=3, head_dim=64, window=50, sinks=4, scale=0.125, dtype=BF16)


def desc(**change):
    return basp.basp_attention_desc(**{**DESC, **change})


def heads(n, length, count, d=64, **change):
    f = dict(data=at(n), stride_batch=length * count * d, stride_seq=count * d, stride_head=d)
    return basp.basp_heads(**{**f, **change})


def forward(lib, d, **change):
    a = dict(q=heads(1, 100, 6), k=heads(2, 300, 3), v=heads(3, 300, 3), o=heads(4, 100, 6), rest=None, lse=at(5))
    return lib.basp_attention(d, *{**a, **change}.values(), None)


DESC_REFUSALS = [
    (dict(batch=-1), INVALID), (dict(q_len=-1), INVALID), (dict(k_len=-1), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(dtype=FP32), INVALID), (dict(dtype=FP8), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=12), INVALID),
    (dict(head_dim=136), INVALID), (dict(q_heads=7), DIVIDE), (dict(k_heads=0), DIVIDE), (dict(q_len=1 << 31), LARGE),
    (dict(batch=1 << 31), LARGE), (dict(batch=1 << 30, q_len=1 << 30), LARGE),
]


@pytest.mark.parametrize("change,status", DESC_REFUSALS)
def test_attention_desc_refusals(lib, change, status):
    d = desc(**change)
    assert forward(lib, d) == status
    assert basp.basp_attention_backward_workspace(d) == 0
    assert basp.basp_attention_decode_workspace(desc(**{**change, "q_len": change.get("q_len", 1)})) == 0 or "q_len" not in change


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(v=heads(3, 300, 3, data=None)), INVALID),
    (dict(q=heads(1, 100, 6, stride_seq=-8)), INVALID), (dict(q=heads(1, 100, 6, data=at(1) + 8)), ALIGN),
    (dict(k=heads(2, 300, 3, stride_seq=196)), ALIGN), (dict(v=heads(3, 300, 3, stride_head=60)), ALIGN),
    (dict(o=heads(4, 100, 6, stride_head=0)), ALIAS), (dict(o=heads(4, 100, 6, stride_seq=64)), ALIAS),
    (dict(o=heads(4, 100, 6, stride_head=56)), ALIAS), (dict(o=heads(1, 100, 6)), ALIAS), (dict(o=heads(2, 100, 6)), ALIAS),
    (dict(rest=heads(4, 100, 6)), ALIAS), (dict(rest=heads(1, 100, 6)), ALIAS), (dict(rest=heads(7, 100, 6, stride_head=0)), ALIAS),
    (dict(rest=heads(7, 100, 6, data=at(7) + 4)), ALIGN), (dict(rest=heads(7, 100, 6, data=None)), INVALID),
    (dict(rest=heads(7, 100, 6, stride_seq=388)), ALIGN),
    (dict(lse=at(4)), ALIAS), (dict(lse=at(5) + 2), ALIGN), (dict(k=heads(2, 300, 3, stride_batch=1 << 57)), LARGE),
])
def test_attention_refusals(lib, change, status):
    assert forward(lib, desc(), **change) == status


def test_attention_of_nothing(lib):
    assert forward(lib, desc(batch=0), q=None, k=None, v=None, o=None) == OK
    assert forward(lib, desc(q_len=0), q=None, o=None) == OK
    assert forward(lib, desc(q_heads=0), q=None, o=None) == OK


@pytest.mark.parametrize("change,status", [
    (dict(d_o=None), INVALID), (dict(lse=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dv=heads(3, 300, 3)), ALIAS), (dict(dk=heads(9, 300, 3)), ALIAS), (dict(dq=heads(4, 100, 6)), ALIAS),
    (dict(dv=heads(9, 300, 3, stride_batch=0)), ALIAS), (dict(ws=None), WORKSPACE), (dict(wsb=1), WORKSPACE),
    (dict(rest=heads(12, 100, 6, data=None)), INVALID), (dict(rest=heads(7, 100, 6)), ALIAS), (dict(rest=heads(11, 100, 6)), ALIAS),
    (dict(ws=at(11) + 8), ALIGN), (dict(ws=at(8)), ALIAS), (dict(dk=heads(8, 300, 3, data=at(8) + 2)), ALIGN),
])
def test_attention_backward_refusals(lib, change, status):
    d = desc()
    a = dict(q=heads(1, 100, 6), k=heads(2, 300, 3), v=heads(3, 300, 3), o=heads(4, 100, 6), rest=None, lse=at(5), d_o=heads(6, 100, 6),
             dq=heads(7, 100, 6), dk=heads(8, 300, 3), dv=heads(9, 300, 3), ws=at(11),
             wsb=basp.basp_attention_backward_workspace(d))
    assert lib.basp_attention_backward(d, *{**a, **change}.values(), None) == status


@pytest.mark.parametrize("change,status", [
    (dict(desc=desc(q_len=2)), INVALID), (dict(desc=desc(q_len=0)), INVALID), (dict(q=None), INVALID), (dict(lengths=None), INVALID),
    (dict(lengths=at(5) + 2), ALIGN), (dict(o=heads(2, 1, 6)), ALIAS), (dict(k=heads(2, 300, 3, data=at(2) + 2)), ALIGN),
])
def test_attention_decode_refusals(lib, change, status):
    d = desc(q_len=1)
    a = dict(desc=d, q=heads(1, 1, 6), k=heads(2, 300, 3), v=heads(3, 300, 3), lengths=at(5), o=heads(4, 1, 6), ws=at(6),
             wsb=max(0, basp.basp_attention_decode_workspace(d)))
    assert lib.basp_attention_decode(*{**a, **change}.values(), None) == status


def adam(place, **change):
    f = dict(p=at(place), g=at(place + 1), m=at(place + 2), v=at(place + 3), m_scales=None, v_scales=None, n=100, dtype=FP32, grad_dtype=FP32)
    return basp.basp_adamw_tensor(**{**f, **change})


def eight(place, **change):
    return adam(place, **{**dict(m_scales=at(place + 4), v_scales=at(place + 5)), **change})


OPTIONS = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, step_at=None, seed=0)


@pytest.mark.parametrize("tensors,change,status", [
    ([], {}, OK), ([adam(1, n=0, p=None, g=None, m=None, v=None)], {}, OK),
    ([adam(1, n=-1)], {}, INVALID), ([adam(1, dtype=FP8)], {}, INVALID), ([adam(1, dtype=BF16, grad_dtype=FP16)], {}, INVALID),
    ([adam(1, dtype=FP32, grad_dtype=BF16)], {}, INVALID), ([adam(1, p=None)], {}, INVALID), ([adam(1, m=None)], {}, INVALID),
    ([adam(1, m_scales=at(9))], {}, INVALID), ([eight(1), adam(10)], {}, INVALID), ([adam(1), eight(10)], {}, INVALID),
    ([adam(1, g=at(2) + 2)], {}, ALIGN), ([adam(1, g=at(1))], {}, ALIAS), ([adam(1, v=at(3))], {}, ALIAS),
    ([eight(1, v_scales=at(5))], {}, ALIAS), ([adam(1, n=1 << 60)], {}, LARGE),
    ([adam(1)], dict(lr=-1.0), INVALID), ([adam(1)], dict(lr=float("nan")), INVALID), ([adam(1)], dict(beta1=1.0), INVALID),
    ([adam(1)], dict(beta2=-0.1), INVALID), ([adam(1)], dict(eps=float("inf")), INVALID), ([adam(1)], dict(step=0), INVALID),
    ([adam(1)], dict(weight_decay=float("nan")), INVALID), ([adam(1)], dict(step=1 << 31), INVALID), ([adam(1)], dict(step_at=at(9) + 2), ALIGN),
])
def test_adamw_refusals(lib, tensors, change, status):
    table = (basp.basp_adamw_tensor * max(1, len(tensors)))(*tensors)
    assert lib.basp_adamw(table, len(tensors), basp.basp_adamw_options(**{**OPTIONS, **change}), None) == status


def test_adamw_pointers(lib):
    o = basp.basp_adamw_options(**OPTIONS)
    assert lib.basp_adamw(None, 1, o, None) == INVALID and lib.basp_adamw(None, 0, o, None) == OK
    assert lib.basp_adamw(None, 0, None, None) == INVALID and lib.basp_adamw(None, -1, o, None) == INVALID
    assert lib.basp_attention_timeouts(None) == INVALID


def test_python_refusals():
    """What the tensors' calls refuse before they look for a GPU."""
    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.ones(16, dtype=torch.bfloat16)
    q, k = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16)
    p = torch.zeros(8)
    for call in (lambda: fp8.layernorm(x, w), lambda: fp8.layernorm(x.double(), w), lambda: fp8.layernorm(x, None),
                 lambda: fp8.layernorm_backward(x, x, torch.ones(4), torch.ones(4), w), lambda: attention.forward(q, k, k),
                 lambda: attention.forward(q.float(), k, k), lambda: attention.forward(q[0], k, k),
                 lambda: attention.forward(q, k, k, window=0), lambda: attention.forward(q, k, k, window=2.5),
                 lambda: attention.forward(q, k, k, sinks=-1), lambda: attention.forward(q, k, k, scale="x"),
                 lambda: attention.forward(q, k, k, scale=float("inf")), lambda: attention.forward(q[..., :60], k, k),
                 lambda: attention.forward(q[:, :, :1], k.expand(1, 4, 2, 64), k), lambda: attention.forward(q, None, k),
                 lambda: attention.decode(q[:, 0], k, k, torch.ones(1, dtype=torch.int32)), lambda: attention.decode(q, k, k, p),
                 lambda: attention.backward(q, q, k, k, q, p), lambda: optim.adamw([p], [p], [p], [], 1),
                 lambda: optim.adamw([p], [], [p], [p], 1), lambda: optim.adamw(p, [p], [p], None, 1),
                 lambda: optim.AdamW([torch.nn.Parameter(p)], state_bits=16), lambda: optim.AdamW([torch.nn.Parameter(p)], lr=-1),
                 lambda: optim.adamw([p], [p], [fp8.Quantized(p, p)], [p], 1)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_torch_module_calls_the_loaded_library(lib):
    names = basp.FP8_EXPORTS[6:] + basp.ATTENTION_EXPORTS[:5] + basp.OPTIM_EXPORTS
    assert list(basp.binding.layer_entry_points()) == [ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names]


# ---- the 64-bit forms themselves ---------------------------------------------------

def test_attention_form_against_torch():
    """One row at a time with torch's own softmax and autograd, in 64 bits."""
    rng = np.random.default_rng(1)
    q, do = rng.standard_normal((9, 4, 8)), rng.standard_normal((9, 4, 8))
    k, v = rng.standard_normal((12, 2, 8)), rng.standard_normal((12, 2, 8))
    a = ref.Attention(q, k, v, 5, 2, 0.3, 0)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    out = torch.zeros(9, 4, 8, dtype=torch.float64)
    for i in range(9):
        keys = [j for j in range(12) if j <= i + 3 and (j > i + 3 - 5 or j < 2)]
        for h in range(4):
            s = 0.3 * tk[keys, h // 2] @ tq[i, h]
            out[i, h] = torch.softmax(s, 0) @ tv[keys, h // 2]
            assert abs(float(torch.logsumexp(s, 0)) - a.lse[h, i]) < 1e-12
    assert np.abs(out.detach().numpy() - a.o).max() < 1e-12
    out.backward(torch.tensor(do))
    grads, bounds = a.backward(do, np.zeros(q.shape))
    for n, t in (("dq", tq), ("dk", tk), ("dv", tv)):
        assert np.abs(t.grad.numpy() - grads[n]).max() < 1e-11 and (bounds[n] < 1e-3).all()


def test_layernorm_form_against_torch():
    rng = np.random.default_rng(2)
    x, w, b, dy, dh = (rng.standard_normal(s) for s in ((5, 33), 33, 33, (5, 33), (5, 33)))
    t = [torch.tensor(y, requires_grad=True) for y in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], 1e-3)
    torch.autograd.backward([y, t[0]], [torch.tensor(dy), torch.tensor(dh)])
    want, mean, rstd = ref.layernorm(x, w, b, 1e-3)
    assert np.abs(y.detach().numpy() - want).max() < 1e-12
    for g, leaf in zip(ref.layernorm_backward(dy, x, mean, rstd, w, dh), t):
        assert np.abs(g - leaf.grad.numpy()).max() < 1e-11


def test_adamw_form_against_torch():
    rng = np.random.default_rng(3)
    p, m, v = rng.standard_normal(50), np.zeros(50), np.zeros(50)
    leaf = torch.tensor(p, requires_grad=True)
    opt = torch.optim.AdamW([leaf], lr=0.02, betas=(0.8, 0.9), eps=1e-3, weight_decay=0.3)
    for step in range(1, 5):
        g = rng.standard_normal(50)
        leaf.grad = torch.tensor(g)
        opt.step()
        p, m, v = ref.adamw(p, g, m, v, step, 0.02, 0.8, 0.9, 1e-3, 0.3)
        assert np.abs(leaf.detach().numpy() - p).max() < 1e-12


def test_random_bits_are_even():
    """The two halves of 2^20 elements' bits, in 64 bins each and in 64 x 64 together:
    chi-squared within six standard deviations; neighbours, steps, seeds and tensors differ."""
    n = 1 << 20
    lo, hi = ref.random_bits(n, 5, 17, 2)
    for bins, counts in ((64, np.bincount((lo >> np.uint64(10)).astype(int), minlength=64)),
                         (64, np.bincount((hi >> np.uint64(10)).astype(int), minlength=64)),
                         (4096, np.bincount((lo >> np.uint64(10)).astype(int) * 64 + (hi >> np.uint64(10)).astype(int), minlength=4096)),
                         (4096, np.bincount((lo[1:] >> np.uint64(10)).astype(int) * 64 + (lo[:-1] >> np.uint64(10)).astype(int), minlength=4096))):
        expected = counts.sum() / bins
        chi = ((counts - expected) ** 2 / expected).sum()
        assert abs(chi - (bins - 1)) <= 6 * np.sqrt(2 * bins)
    for other in (ref.random_bits(n, 6, 17, 2), ref.random_bits(n, 5, 18, 2), ref.random_bits(n, 5, 17, 3)):
        a, b = lo.astype(float) - 32767.5, other[0].astype(float) - 32767.5
        assert abs((a * b).mean() / (65536 ** 2 / 12)) <= 6 / np.sqrt(n)


@pytest.mark.parametrize("places,status", [
    ([1, 10, 1], ALIAS), ([1, 1], ALIAS), ([30, 20, 10, 20], ALIAS), (list(range(10, 10 + 6 * 600, 6)) + [10], ALIAS)])
def test_a_parameter_does_not_come_twice(lib, places, status):
    table = (basp.basp_adamw_tensor * len(places))(*(adam(p, g=at(9000), m=at(9001), v=at(9002)) for p in places))
    assert lib.basp_adamw(table, len(places), basp.basp_adamw_options(**OPTIONS), None) == status
    part = adam(1, p=at(1) + 396, g=at(9000), m=at(9001), v=at(9002))
    assert lib.basp_adamw((basp.basp_adamw_tensor * 2)(adam(1), part), 2, basp.basp_adamw_options(**OPTIONS), None) == ALIAS


@pytest.mark.parametrize("name", ["q_len", "k_len"])
def test_the_longest_sequences(lib, name):
    """A loop over a sequence steps past its end: lengths leave room below 2^31."""
    assert forward(lib, desc(**{name: 2 ** 31 - 4095})) == LARGE
    assert basp.basp_attention_decode_workspace(desc(q_len=1, k_len=2 ** 31 - 4095, window=0)) == 0
    assert basp.basp_attention_decode_workspace(desc(q_len=1, k_len=2 ** 31 - 4096, window=0)) > 0


@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_parameters_count_the_steps_they_take(capturable, bits, monkeypatch):
    """As torch.optim.AdamW's; also from a saved state on in which two numbers were equal by chance."""
    taken = []

    def call(params, grads, m, v, step, *rest):
        taken.append([int(s) for s in step] if isinstance(step, list) else [step] * len(params))

    monkeypatch.setattr(optim, "adamw", call)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    params = [torch.nn.Parameter(torch.zeros(3)) for _ in range(3)]
    mine = optim.AdamW(params, capturable=capturable, state_bits=bits)
    theirs = torch.optim.AdamW(params)
    # the second misses steps 2 to 5, the third joins in step 4 and misses step 8
    has = [(1, 1, 0), (1, 0, 0), (1, 0, 0), (1, 0, 1), (1, 0, 1), (1, 1, 1), (1, 1, 1), (1, 1, 0), (1, 1, 1)]
    for i, h in enumerate(has):
        if i == 7:
            old = mine
            numbers = [int(old.state[p]["step"]) for p in params]
            assert numbers == [7, 3, 4]
            for p in params:                              # equal by chance
                old.state[p]["step"] = torch.full((1,), 4, dtype=torch.int32) if capturable else 4
            mine = optim.AdamW(params, capturable=capturable, state_bits=bits)
            mine.load_state_dict(old.state_dict())
            want = [4, 4, 4]
        for p, x in zip(params, h):
            p.grad = torch.ones(3) if x else None
        taken.clear()
        mine.step()
        if i < 7:
            theirs.step()
            want = [int(theirs.state[p]["step"]) if p in theirs.state else None for p in params]
        else:
            want = [w + x for w, x in zip(want, h)]
        assert [int(mine.state[p]["step"]) if mine.state.get(p) else None for p in params] == want
        assert sorted(n for t in taken for n in t) == sorted(w for w, x in zip(want, h) if x)


def test_numbers_of_steps_of_their_own(lib):
    def status(tensors, steps, **change):
        table, at = (basp.basp_adamw_tensor * len(tensors))(*tensors), (ctypes.c_void_p * len(tensors))(*steps)
        return lib.basp_adamw_each(table, at, None, len(tensors), basp.basp_adamw_options(**{**OPTIONS, "step": 0, **change}), None)
    assert status([adam(1)], [at(90) + 2]) == ALIGN and status([adam(1, n=0)], [at(90) + 2]) == ALIGN
    assert status([adam(1), adam(10)], [at(90), None]) == INVALID and status([adam(1, p=None)], [at(90)]) == INVALID
    assert status([adam(1, n=0)], [None]) == OK and status([], []) == OK
    assert status([adam(1), adam(1)], [at(90), at(91)]) == ALIAS and status([adam(1)], [at(90)], lr=-1.0) == INVALID
    o = basp.basp_adamw_options(**OPTIONS)
    assert lib.basp_adamw_each((basp.basp_adamw_tensor * 1)(adam(1, p=None)), None, None, 1, o, None) == INVALID
    assert lib.basp_adamw_each(None, None, None, 0, o, None) == OK and lib.basp_adamw_each(None, None, None, -1, o, None) == INVALID
    o.step = 0
    assert lib.basp_adamw_each(None, None, None, 0, o, None) == INVALID
    for change in (dict(steps_at=[]), dict(steps_at=None, numbers=[])):
        with pytest.raises(ValueError):
            basp.basp_adamw_each([adam(1)], options=o, **change)


@pytest.mark.parametrize("offset", [0, 1, 3, 4, 8, 16])
def test_gradients_that_begin_anywhere(offset):
    """What the attention's backward gets begins at a multiple of 16 bytes, also of a piece that is contiguous."""
    flat = torch.arange(2 * 5 * 3 * 8 + 40, dtype=torch.float32).bfloat16()
    flat = flat[(-flat.data_ptr() // 2) % 8:]
    t = flat[offset:offset + 240].view(2, 5, 3, 8)
    got = autograd._aligned(t)
    assert t.is_contiguous() and got.data_ptr() % 16 == 0 and torch.equal(got, t)
    assert (got is t) == (offset % 8 == 0)
    for spread in (t[:, :1].expand(2, 5, 3, 8), t.transpose(0, 1), t[..., :1].expand(2, 5, 3, 8), t[:1, :, :, :4].expand(2, 5, 3, 4)):
        got = autograd._aligned(spread)
        assert got.data_ptr() % 16 == 0 and torch.equal(got, spread) and got.stride(-1) == 1
        assert all(s % 8 == 0 for s, n in zip(got.stride()[:-1], got.shape) if n > 1) or spread.shape[-1] == 4


@pytest.mark.parametrize("bad", [dict(state_bits=16), dict(lr=-1.0), dict(lr=float("nan")), dict(eps=-1e-8), dict(weight_decay=-0.1),
                                 dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(betas=(0.9,))])
def test_options_of_a_group(bad):
    """A group's own options are refused as the constructor's are, and the group is not taken."""
    a, b = (torch.nn.Parameter(torch.zeros(3)) for _ in range(2))
    with pytest.raises(ValueError):
        optim.AdamW([a], **bad)
    with pytest.raises(ValueError):
        optim.AdamW([{"params": [a], **bad}])
    o = optim.AdamW([a])
    with pytest.raises(ValueError):
        o.add_param_group({"params": [b], **bad})
    assert len(o.param_groups) == 1
    o.add_param_group({"params": [b], "state_bits": 8, "lr": 0.0})
    assert [g["state_bits"] for g in o.param_groups] == [32, 8]
    with pytest.raises(TypeError):
        o.add_param_group([b])


@pytest.mark.parametrize("change,status", DESC_REFUSALS)
def test_workspaces_of_what_is_refused(lib, change, status):
    """A call that is refused needs none; only a bad q_len alone is a good decode call without it."""
    one = basp.basp_attention_decode_workspace(desc(**{"window": 0, "k_len": 100000, **change, "q_len": 1}))
    assert (one > 0) == (set(change) == {"q_len"})
    if "q_len" in change:
        assert basp.basp_attention_decode_workspace(desc(**change)) == 0
    assert basp.basp_attention_backward_workspace(desc(**change)) == 0
