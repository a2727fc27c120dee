"""AdamW over many tensors (include/basp_optim.h) against its 64-bit form.

Tolerances.  A rounding of m' is 3 * 2^-24 of the magnitudes it adds, of v' 4 * 2^-24 of
itself; the quotient has the root's half of that, c1's and c2's 2^-24 each and a
division good to 2^-22: 2^-20 of the step in all, and p's own roundings (the decay's
factor, the sum, and its type's)."""
import numpy as np
import pytest
import torch

import fp8_reference as ref8
import layer_reference as ref
from sequence_re_layout_gb300 import fp8, optim

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F32, TINY = ref.F32, ref.TINY
BETAS, EPS = (0.9, 0.999), 1e-8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sequence_re_layout_gb300.build import build_library
    build_library()


def u(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def random(n, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * scale).to(dtype).cuda()


def spread(n, seed):
    """Magnitudes over several powers of ten."""
    g = torch.Generator().manual_seed(seed)
    return torch.exp(2 * torch.randn(n, generator=g) - 6).cuda()


def check(p, g, m, v, got, step, lr, wd):
    """(p', m', v') of 64 bits, the kernel's against them; m and v as the kernel had them."""
    p1, m1, v1 = ref.adamw(f64(p), f64(g), m, v, step, lr, *BETAS, EPS, wd)
    up = np.abs(p1 - f64(p) * (1 - lr * wd))
    em = 4 * F32 * (np.abs(m) + np.abs(f64(g)))
    room = lr / (1 - BETAS[0] ** step) * em / (np.sqrt(v1) / np.sqrt(1 - BETAS[1] ** step) + EPS)
    bound = 2.0 ** -20 * up + 2 * room + 3 * F32 * np.abs(f64(p)) + TINY
    assert (np.abs(f64(got) - p1) <= bound + u(got.dtype) * (np.abs(p1) + bound)).all()
    return m1, v1, em


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("grad32", [False, True])
@pytest.mark.parametrize("step", [1, 2, 1000, 2 ** 31 - 1])
def test_32_bits(dtype, grad32, step):
    t = DTYPES[dtype]
    sizes = [1, 3, 4, 127, 128, 129, 512, 1000, 4096, 16384, 16385, 50000, 0]
    p = [random(n, t, 3 * i) for i, n in enumerate(sizes)]
    g = [(random(n, torch.float32, 3 * i + 1) * spread(n, i)).to(torch.float32 if grad32 else t) for i, n in enumerate(sizes)]
    m = [random(n, torch.float32, 3 * i + 2) * spread(n, i) for i, n in enumerate(sizes)]
    v = [(spread(n, i + 50)) ** 2 for i, n in enumerate(sizes)]
    old = [[x.clone() for x in xs] for xs in (p, m, v)]
    optim.adamw(p, g, m, v, step, lr=0.01, weight_decay=0.1)
    for i in range(len(sizes)):
        m1, v1, em = check(old[0][i], g[i], f64(old[1][i]), f64(old[2][i]), p[i], step, 0.01, 0.1)
        assert (np.abs(f64(m[i]) - m1) <= em + TINY * 2.0 ** -100).all()
        assert (np.abs(f64(v[i]) - v1) <= 6 * F32 * v1 + 2.0 ** -148).all()


def quantized(values):
    """[1, n] in 8 bits, as a state."""
    return fp8.quantize(values.view(1, -1).float())


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("step,seed", [(1, 0), (7, 123456789), (2 ** 31 - 1, 2 ** 32 - 1)])
def test_8_bits(dtype, step, seed):
    t = DTYPES[dtype]
    sizes = [1, 3, 127, 128, 129, 130, 1000, 4096, 16384, 16390, 50000]
    p = [random(n, t, 3 * i) for i, n in enumerate(sizes)]
    g = [(random(n, torch.float32, 3 * i + 1) * spread(n, i)).to(t) for i, n in enumerate(sizes)]
    m = [quantized(random(n, torch.float32, 3 * i + 2) * spread(n, i)) for i, n in enumerate(sizes)]
    v = [quantized(spread(n, i + 50)) for i, n in enumerate(sizes)]
    old_p, old_m, old_r = [x.clone() for x in p], [f64(x.dequantize())[0] for x in m], [f64(x.dequantize())[0] for x in v]
    optim.adamw(p, g, m, v, step, lr=0.01, weight_decay=0.1, seed=seed)
    flips = total = 0
    for i, n in enumerate(sizes):
        m1, v1, em = check(old_p[i], g[i], old_m[i], old_r[i] ** 2, p[i], step, 0.01, 0.1)
        for q, want, error, r in ((m[i], m1, em, 0), (v[i], np.sqrt(v1), 4 * F32 * np.sqrt(v1), 1)):
            e = q.scales.cpu().view(torch.uint8).numpy().astype(np.int64)[0] - 127
            exps = ref8.quantize(want[None], 1)[1][0]
            blocks = np.arange(n) // 128
            same = (e == exps)[blocks]                     # a block's maximum next to a power's end may go either way
            assert (np.abs(e - exps) <= 1).all() and (e != exps).mean() <= 0.02
            scale = 2.0 ** e[blocks].astype(np.float64)
            y, room = ref.round_at_random(want / scale, ref.random_bits(n, seed, step, i)[r])
            got = f64(q.data.float())[0]
            if r:
                y = np.where((want > 0) & (y == 0), 2.0 ** -9, y)
            steps = error / scale / 2.0 ** (np.maximum(np.frexp(np.abs(want / scale))[1] - 1, -6) - 3)
            sure = same & (room > steps + 2.0 ** -18)      # 32 bits decide as 64 do
            assert np.array_equal(got[sure], y[sure])
            assert sure[same].mean() > 0.9 or n < 200
            step_up = 2.0 ** -3 * np.abs(want) + 2.0 ** -9 * scale + 2 * error
            assert (np.abs(got * scale - want) <= step_up).all()


def test_the_rounding_is_fair():
    """The mean over many elements is the value: each is up with the fraction's
    probability.  2^20 draws: six standard deviations of sqrt(1/4 / 2^20) steps."""
    n = 1 << 20
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for value in (0.3, 1.0, 2.0 ** -9 * 0.4, 100.0):
        m = quantized(torch.full((n,), 448.0, device="cuda"))
        v = quantized(torch.full((n,), 448.0, device="cuda"))
        g.fill_(0.0)
        # m' = 0.9 * 448 in a block whose largest is 448: the block's first keeps the scale
        g[:] = (value - 0.9 * 448) / 0.1
        g[::128] = 448.0
        optim.adamw([p], [g], [m], [v], 5, lr=0.0, weight_decay=0.0, seed=7)
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[::128] = False
        want = 0.9 * 448 + 0.1 * float(g[1])
        got = m.dequantize()[0][rest].double()
        step = float(2.0 ** (max(np.floor(np.log2(value)), -6) - 3))
        assert abs(float(got.mean()) - want) <= 6 * 0.5 * step / np.sqrt(n * 127 / 128) + 2.0 ** -16 * 448 * 2.0 ** -6
        # m' is off by roundings of 0.9 * 448: next to a power of two it may be below it, where steps are half as wide
        grid = step / 2 if np.log2(value) == np.floor(np.log2(value)) else step
        assert set(np.unique(f64(got) / grid % 1)) == {0.0}


def test_small_changes_of_v_are_not_lost():
    """A gradient of zero for 700 steps: v falls by 0.999^700, its root by half of that
    in the logarithm.  The mean of 2^16 roots, each a walk whose steps have a spread of at
    most 2^-4 of the value: six standard deviations."""
    n = 1 << 16
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = quantized(torch.zeros(n, device="cuda")), quantized(torch.full((n,), 1.0, device="cuda"))
    g[::128] = 1.0                                          # keeps the blocks' scale
    for step in range(1, 701):
        optim.adamw([p], [g], [m], [v], step, lr=0.0)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::128] = False
    got = float(v.dequantize()[0][rest].double().mean())
    want = 0.999 ** 350
    assert abs(got / want - 1) <= 6 * 2.0 ** -4 * np.sqrt(700 * 0.01) / np.sqrt(n) + 0.01


def test_many_tensors_and_types_in_one_call():
    """More tensors than a launch's table has; mixed types; the result is that of one call each."""
    n_of = lambda i: 1 + i * 37 % 999                       # noqa: E731
    types = [torch.float32, torch.bfloat16, torch.float16]
    make = lambda: ([random(n_of(i), types[i % 3], i) for i in range(1100)],            # noqa: E731
                    [random(n_of(i), types[i % 3] if i % 2 else torch.float32, i + 5000) for i in range(1100)],
                    [random(n_of(i), torch.float32, i + 9000) for i in range(1100)],
                    [random(n_of(i), torch.float32, i + 7000).square() for i in range(1100)])
    a, b = make(), make()
    optim.adamw(*a, step=3)
    for i in range(1100):
        optim.adamw(*([x[i]] for x in b), step=3)
    for x, y in zip(a, b):
        assert all(torch.equal(s, t) for s, t in zip(x, y))


def test_places():
    """Pieces of one buffer that begin anywhere; nothing beside them is written."""
    store = torch.zeros(4000, device="cuda")
    p, g, m, v = (random(4000, torch.float32, s) for s in range(4))
    v = v.square()
    whole = [x.clone() for x in (p, m, v)]
    optim.adamw([whole[0]], [g], [whole[1]], [whole[2]], 4)
    cuts = [0, 1, 6, 131, 132, 517, 1544, 3999]
    parts = [[x[i:j] for i, j in zip(cuts, cuts[1:])] for x in (p, g, m, v)]
    last = [x[3999:].clone() for x in (p, m, v)]
    optim.adamw(*parts, step=4)
    for x, y, z in zip((p, m, v), whole, last):
        assert torch.equal(x[:3999], y[:3999]) and torch.equal(x[3999:], z)
    assert bool((store == 0).all())


def test_step_on_the_gpu_and_captured():
    p, g, m, v = (random(5000, torch.float32, s) for s in range(4))
    v = v.square()
    q = [x.clone() for x in (p, m, v)]
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(1, 4):
        optim.adamw([p], [g], [m], [v], t)
        step += 1
        optim.adamw([q[0]], [g], [q[1]], [q[2]], step)
        for a, b in zip((p, m, v), q):
            assert bool(((a - b).abs() <= 2.0 ** -20 * a.abs() + 1e-9).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        optim.adamw([q[0]], [g], [q[1]], [q[2]], step)
    for t in range(4, 7):
        optim.adamw([p], [g], [m], [v], t)
        graph.replay()
        torch.cuda.synchronize()
        assert int(step) == t
        for a, b in zip((p, m, v), q):
            assert bool(((a - b).abs() <= 2.0 ** -20 * a.abs() + 1e-9).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_no_number(bits, bad):
    """It stays in its element (and with 8 bits, does not touch the block's scale)."""
    def make():
        p, g = random(300, torch.float32, 1), random(300, torch.float32, 2)
        m, v = random(300, torch.float32, 3), random(300, torch.float32, 4).square()
        return p, g, m if bits == 32 else quantized(m), v if bits == 32 else quantized(v.sqrt())
    values = lambda s: (s if bits == 32 else s.dequantize()).view(-1)         # noqa: E731
    p, g, m, v = make()
    optim.adamw([p], [g], [m], [v], 3)
    p2, g2, m2, v2 = make()
    g2[130] = bad
    optim.adamw([p2], [g2], [m2], [v2], 3)
    rest = torch.arange(300, device="cuda") != 130
    for a, b in ((p, p2), (values(m), values(m2)), (values(v), values(v2))):
        assert torch.equal(a[rest], b[rest])
    assert not bool(torch.isfinite(values(m2)[130])) and (bad == bad or bool(torch.isnan(p2[130])))


def test_zeros_stay_zero():
    for bits in (32, 8):
        z = torch.zeros(200, device="cuda")
        m, v = (z.clone(), z.clone()) if bits == 32 else (quantized(z), quantized(z))
        p = random(200, torch.float32, 1)
        old = p.clone()
        optim.adamw([p], [z], [m], [v], 1, lr=0.1, weight_decay=0.0)
        assert torch.equal(p, old)


def layer(seed):
    torch.manual_seed(seed)
    return torch.nn.Sequential(torch.nn.Linear(40, 70), torch.nn.Linear(70, 9)).cuda()


@pytest.mark.parametrize("capturable", [False, True])
def test_optimizer_against_torch(capturable):
    """torch.optim.AdamW in 64 bits; 20 steps of rounding 2^-20 of a step's size."""
    a, b = layer(1), layer(1).double()
    mine = optim.AdamW(a.parameters(), lr=0.01, weight_decay=0.2, capturable=capturable)
    theirs = torch.optim.AdamW(b.parameters(), lr=0.01, weight_decay=0.2)
    for i in range(20):
        for x, y in zip(a.parameters(), b.parameters()):
            x.grad = random(x.numel(), torch.float32, 100 * i + x.numel() % 97).view_as(x)
            y.grad = x.grad.double()
        mine.step()
        theirs.step()
    for x, y in zip(a.parameters(), b.parameters()):
        assert bool(((x.double() - y).abs() <= 20 * (0.02 * 2.0 ** -18 + 2.0 ** -23 * y.abs())).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_optimizer_resumes(bits, capturable):
    """Ten steps are five, a saved state, and five more: bit for bit; also parameters that join later."""
    def run(resume):
        net = layer(2).bfloat16()
        opt = optim.AdamW(net.parameters(), lr=0.01, state_bits=bits, capturable=capturable, seed=3)
        for i in range(10):
            for j, p in enumerate(net.parameters()):
                p.grad = random(p.numel(), torch.bfloat16, 10 * i + j).view_as(p) if j < 2 or i > 2 else None
            opt.step()
            if resume and i == 4:
                saved = opt.state_dict()
                opt = optim.AdamW(net.parameters(), lr=0.5, state_bits=bits, capturable=capturable, seed=9)
                opt.load_state_dict(saved)
        return net, opt
    (a, oa), (b, ob) = run(False), run(True)
    assert all(torch.equal(x, y) for x, y in zip(a.parameters(), b.parameters()))
    steps = [int(oa.state[p]["step"]) for p in a.parameters()]
    assert steps == [10, 10, 7, 7] == [int(ob.state[p]["step"]) for p in b.parameters()]


def test_optimizer_captured():
    nets = [layer(3), layer(3)]
    opts = [optim.AdamW(n.parameters(), lr=0.01, state_bits=8, capturable=True) for n in nets]
    grads = [random(p.numel(), torch.float32, i).view_as(p) for i, p in enumerate(nets[0].parameters())]
    for n, o in zip(nets, opts):
        for p, g in zip(n.parameters(), grads):
            p.grad = g.clone()
        o.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opts[1].step()
    for _ in range(3):
        opts[0].step()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(nets[0].parameters(), nets[1].parameters()))
    plain = optim.AdamW(nets[0].parameters())
    plain.step()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="capturable"):
        with torch.cuda.graph(graph):
            plain.step()


def test_autograd_is_told():
    w = torch.randn(64, device="cuda", requires_grad=True)
    y = torch.exp(w)
    w.grad = torch.ones_like(w)
    opt = optim.AdamW([w])
    z = w * w
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    del y


@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_tiny_gradients_without_eps(dtype):
    """v below 2^-126: its root is not, and the step is lr by the first one's definition."""
    n = 1000
    g = (random(n, torch.float32, 3).sign() * 2.0 ** -60)
    p = torch.ones(n, dtype=DTYPES[dtype], device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    optim.adamw([p], [g], [m], [v], 1, lr=0.5, eps=0.0, weight_decay=0.0)
    # v' = 0.001 * 2^-120 is a multiple of 2^-149: off by 2^-150, 2^-20 of it, its root by half of that
    want, t = 1 - 0.5 * f64(g.sign()), DTYPES[dtype]
    assert bool((v > 0).all()) and (np.abs(f64(p) - want) <= 0.5 * 2.0 ** -20 + u(t) * 2).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_first_step_is_not_captured(bits):
    """Its states would be made anew by every replay."""
    p = torch.nn.Parameter(torch.ones(300, device="cuda"))
    p.grad = torch.ones_like(p)
    o = optim.AdamW([p], state_bits=bits, capturable=True)
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            o.step()
    torch.cuda.synchronize()
    assert bool((p == 1).all()) and not o.state.get(p)
    o.step()
    torch.cuda.synchronize()
    assert bool((p < 1).all()) and int(o.state[p]["step"]) == 1


def test_a_parameter_does_not_come_twice():
    p, g, m, v = (torch.ones(200, device="cuda") for _ in range(4))
    with pytest.raises((ValueError, RuntimeError), match="overlap|alias"):
        optim.adamw([p, p], [g, g], [m, m.clone()], [v, v.clone()], 1)
    assert bool((p == 1).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_a_number_for_each_tensor(bits):
    """More tensors than a launch's table has: each as with its number for all."""
    numbers = [1 + i * i % 50 for i in range(900)]
    def make():
        p, g = ([random(1 + i % 300, torch.float32, i + s) for i in range(900)] for s in (0, 1000))
        m, v = ([random(1 + i % 300, torch.float32, i + s).square() for i in range(900)] for s in (2000, 3000))
        return (p, g, m, v) if bits == 32 else (p, g, [quantized(x) for x in m], [quantized(x.sqrt()) for x in v])
    values = lambda s: s if bits == 32 else s.dequantize()                    # noqa: E731
    a = make()
    steps = list(torch.tensor(numbers, dtype=torch.int32, device="cuda").split(1))
    optim.adamw(*a, step=steps, seed=5)
    one = {}
    for n in sorted(set(numbers)):                          # the whole list with that number
        b = make()
        optim.adamw(*b, step=torch.full((1,), n, dtype=torch.int32, device="cuda"), seed=5)
        one[n] = b
    for i, n in enumerate(numbers):
        for x, y in ((a[0][i], one[n][0][i]), (values(a[2][i]), values(one[n][2][i])), (values(a[3][i]), values(one[n][3][i]))):
            assert torch.equal(x, y)
    for bad in (steps[:-1], [s.long() for s in steps], [s.cpu() for s in steps], numbers):
        with pytest.raises(ValueError):
            optim.adamw(*a, step=bad)


@pytest.mark.parametrize("capturable", [False, True])
def test_parameters_that_miss_steps(capturable):
    """torch.optim.AdamW in 64 bits, where a parameter has no gradient in some steps."""
    a, b = layer(1), layer(1).double()
    mine = optim.AdamW(a.parameters(), lr=0.01, weight_decay=0.2, capturable=capturable)
    theirs = torch.optim.AdamW(b.parameters(), lr=0.01, weight_decay=0.2)
    for i in range(20):
        for j, (x, y) in enumerate(zip(a.parameters(), b.parameters())):
            x.grad = random(x.numel(), torch.float32, 100 * i + j).view_as(x) if i % (j + 1) == 0 else None
            y.grad = None if x.grad is None else x.grad.double()
        mine.step()
        theirs.step()
    for x, y in zip(a.parameters(), b.parameters()):
        assert int(mine.state[x]["step"]) == int(theirs.state[y]["step"])
        assert bool(((x.double() - y).abs() <= 20 * (0.02 * 2.0 ** -18 + 2.0 ** -23 * y.abs())).all())


def test_captured_steps_of_some_and_of_all():
    """Two graphs, one of whose steps leaves parameters out, and plain steps between them."""
    nets = [layer(3), layer(3)]
    opts = [optim.AdamW(n.parameters(), lr=0.01, capturable=c) for n, c in zip(nets, (True, False))]
    def grads(net, every):
        for j, p in enumerate(net.parameters()):
            p.grad = random(p.numel(), torch.float32, j).view_as(p) if every or j % 2 else None
    graphs = []
    grads(nets[0], True)
    opts[0].step()
    keep = []                                               # the gradients that the graphs read
    for every in (True, False):
        grads(nets[0], every)
        keep.append([p.grad for p in nets[0].parameters()])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            opts[0].step()
    for every in (False, False, True, False, True):
        graphs[0 if every else 1].replay()
    grads(nets[0], False)
    opts[0].step()
    for every in (True, False, False, True, False, True, False):
        grads(nets[1], every)
        opts[1].step()
    for x, y in zip(nets[0].parameters(), nets[1].parameters()):
        assert int(opts[0].state[x]["step"]) == opts[1].state[y]["step"]
        assert bool(((x - y).abs() <= 7 * (0.02 * 2.0 ** -18 + 2.0 ** -23 * y.abs())).all())


def test_numbers_of_the_tensors():
    """The bits follow a tensor's number, not its place in the list."""
    def make():
        p, g = ([random(777, torch.float32, i + s) for i in range(5)] for s in (0, 10))
        m, v = ([quantized(random(777, torch.float32, i + s).abs()) for i in range(5)] for s in (20, 30))
        return p, g, m, v
    a, b, c = make(), make(), make()
    optim.adamw(*a, step=3, seed=2)
    order = [3, 0, 4, 2, 1]
    optim.adamw(*([x[i] for i in order] for x in b), step=3, seed=2, numbers=order)
    for x, y in zip(a[2] + a[3], b[2] + b[3]):
        assert torch.equal(x.dequantize(), y.dequantize())
    optim.adamw(*c, step=3, seed=2, numbers=[1000, 2 ** 32 - 1, 7, 6, 5])
    for x, y, number in ((a, c, 0),):
        assert all(torch.equal(s, t) for s, t in zip(x[0], y[0]))       # the step is made before the rounding
        assert not any(torch.equal(s.dequantize(), t.dequantize()) for s, t in zip(x[2] + x[3], y[2] + y[3]))
    for bad in ([1, 2], [1, 2, 3, 4, "5"], [0, 1, 2, 3, -1], 5):
        with pytest.raises(ValueError):
            optim.adamw(*a, step=4, numbers=bad)


@pytest.mark.parametrize("capturable", [False, True])
def test_bits_of_groups_and_of_missing_gradients(capturable):
    """Equal parameters of two groups are rounded by bits of their own, and a parameter's bits do
    not depend on whether one before it has a gradient."""
    def run(first):
        ps = [torch.nn.Parameter(random(2000, torch.float32, s)) for s in (1, 2, 1, 2)]
        o = optim.AdamW([{"params": ps[:2]}, {"params": ps[2:]}], state_bits=8, seed=3, capturable=capturable)
        for i in range(3):
            for j, p in enumerate(ps):
                p.grad = random(2000, torch.float32, 10 * i + j % 2) if first or j % 2 else None
            o.step()
        return [(o.state[p]["exp_avg"].float(), o.state[p]["exp_avg_sq_root"].float()) if o.state.get(p) else None for p in ps]
    a, b = run(True), run(False)
    for i in (0, 1):
        assert not torch.equal(a[0][i], a[2][i]) and not torch.equal(a[1][i], a[3][i])
        assert torch.equal(a[1][i], b[1][i]) and torch.equal(a[3][i], b[3][i])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
def test_nothing_is_written_beside_the_tensors(offset, dtype, bits):
    """Every buffer lies in a larger one, whose other elements stay as they were."""
    t, guard = DTYPES[dtype], 40
    for n in (1, 3, 4, 127, 128, 130, 517, 4096, 16390):
        def inside(values, fill):
            whole = torch.full((n_of(values) + 2 * guard,), fill, dtype=values.dtype, device="cuda")
            at = (guard & ~15) + offset
            whole[at:at + n_of(values)] = values.view(-1)
            return whole, whole[at:at + n_of(values)].view(values.shape), at
        n_of = lambda x: x.numel()                            # noqa: E731
        p, g = random(n, t, 1), random(n, t, 2)
        m, v = random(n, torch.float32, 3), random(n, torch.float32, 4).square()
        if bits == 32:
            want = [p.clone(), g, m.clone(), v.clone()]
            optim.adamw(*([x] for x in want), step=3)
            places = [inside(x, 7.0) for x in (p, g, m, v)]
            optim.adamw(*([x[1]] for x in places), step=3)
        else:
            m, v = quantized(m), quantized(v.sqrt())
            want = [p.clone(), g, m.data.clone(), m.scales.clone(), v.data.clone(), v.scales.clone()]
            state = [fp8.Quantized(want[2], want[3]), fp8.Quantized(want[4], want[5])]
            optim.adamw([want[0]], [g], [state[0]], [state[1]], step=3)
            want = [x.view(torch.uint8) if x.element_size() == 1 else x for x in want]
            places = [inside(x, 7.0) for x in (p, g)] + [inside(x.view(torch.uint8), 7) for x in (m.data, m.scales, v.data, v.scales)]
            as8 = lambda i, ty: places[i][1].view(1, -1).view(ty)          # noqa: E731
            e4m3, e8m0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
            optim.adamw([places[0][1]], [places[1][1]], [fp8.Quantized(as8(2, e4m3), as8(3, e8m0))],
                        [fp8.Quantized(as8(4, e4m3), as8(5, e8m0))], step=3)
        for x, (whole, part, at) in zip(want, places):
            assert torch.equal(part.view(-1), x.view(-1))
            assert bool((whole[:at] == 7).all()) and bool((whole[at + x.numel():] == 7).all())
