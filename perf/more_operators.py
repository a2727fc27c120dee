"""The rest of a sequence-parallel layer's training step, as measurable cases.

Between the two re-layouts the layer attends, before its projections it may take a norm with a mean,
and after the backward pass its weights take a step:

  attention      causal attention with a sliding window and a few first tokens that stay visible
                 (sinks): the forward pass, or the forward and the backward pass
  decode         the same for one new token of each sequence over a cache
  layernorm      residual addition and layer norm, output in 8 bits with a scale for each 128 values of
                 a row; or its gradient for the residual stream, the weight and the bias
  adamw          a step of Adam with decoupled weight decay over many tensors, its two states in 32
                 bits or in 8

Query i of Sq stands at position p = i + Sk - Sq among the Sk keys and sees key j if j <= p and
(j > p - window or j < sinks).  8-bit values are e4m3; scales are powers of two (e8m0).  With ``own``
false, ``run`` computes each one from elementary torch operations in 32 bits; with ``own`` true it calls
this package.
"""
import math

import torch

own = False

BLOCK = 128           # values that share a scale
E4M3_MAX = 448.0
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ADAM = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.1, "step": 10, "seed": 1234}


def listed():
    return [
        # two sequences of 16384 tokens through one layer without gradients
        {"name": "attention_long", "op": "attention", "B": 2, "Sq": 16384, "Sk": 16384, "Hq": 16, "Hkv": 16,
         "d": 128, "window": 4096, "sinks": 4, "dtype": "bf16", "backward": False},
        # a piece of a prompt behind what is already in the cache; odd sizes on every side
        {"name": "attention_piece", "op": "attention", "B": 3, "Sq": 777, "Sk": 1999, "Hq": 9, "Hkv": 3,
         "d": 80, "window": 0, "sinks": 0, "dtype": "fp16", "backward": False},
        # training at 8192 tokens with shared key heads
        {"name": "attention_train_long", "op": "attention", "B": 2, "Sq": 8192, "Sk": 8192, "Hq": 32, "Hkv": 8,
         "d": 64, "window": 1024, "sinks": 4, "dtype": "bf16", "backward": True},
        # a short fine-tuning batch of odd length
        {"name": "attention_train_ragged", "op": "attention", "B": 2, "Sq": 1021, "Sk": 1021, "Hq": 6, "Hkv": 2,
         "d": 96, "window": 200, "sinks": 7, "dtype": "fp16", "backward": True},
        # one user's next token after a long prompt: what counts is latency
        {"name": "decode_one", "op": "decode", "B": 1, "capacity": 16384, "shortest": 16001, "Hq": 32, "Hkv": 8,
         "d": 64, "window": 0, "sinks": 0, "dtype": "bf16"},
        # a batch of conversations of very different lengths
        {"name": "decode_batch", "op": "decode", "B": 32, "capacity": 16384, "shortest": 1, "Hq": 16, "Hkv": 16,
         "d": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # one decoded token of a hidden size of 16 heads x 128
        {"name": "layernorm_token", "op": "layernorm", "M": 1, "H": 2048, "dtype": "bf16", "backward": False},
        # two sequences of 16384 tokens through one layer
        {"name": "layernorm_long", "op": "layernorm", "M": 32768, "H": 2048, "dtype": "bf16", "backward": False},
        # the same on the way back, with the residual stream's own gradient joining
        {"name": "layernorm_backward_long", "op": "layernorm", "M": 32768, "H": 2048, "dtype": "bf16",
         "backward": True},
        # 32-bit master weights of one layer (packed projection, output projection, four times wider inner layer)
        {"name": "adamw_layer", "op": "adamw", "sizes": "layers", "count": 1, "width": 2048, "dtype": "fp32",
         "bits": 32},
        # four such layers with the states in 8 bits
        {"name": "adamw_layers_8bit", "op": "adamw", "sizes": "layers", "count": 4, "width": 2048, "dtype": "fp32",
         "bits": 8},
        # many small tensors of odd sizes, as adapters and norms have them: what counts is launches
        {"name": "adamw_small", "op": "adamw", "sizes": "ragged", "count": 300, "width": 999, "dtype": "bf16",
         "bits": 32},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    return Hkv * rng.choice([1, 1, 2, 3, 4, 8]), Hkv


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "decode", "decode", "layernorm", "layernorm", "adamw", "adamw"])
    if op in ("attention", "decode"):
        Hq, Hkv = _heads(rng)
        d = rng.choice([64, 128, 64, 128, 32, 40, 72, 80, 96, 112])
        case = {"op": op, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
                "window": rng.choice([0, 1, 2, 2]), "sinks": rng.choice([0, 1, 4, 4, 7, 64, 150])}
        if op == "decode":
            case["capacity"] = _log_int(rng, 1, 40000)
            case["B"] = _log_int(rng, 1, max(1, min(64, (1 << 29) // (case["capacity"] * Hkv * d))))
            case["shortest"] = rng.choice([1, case["capacity"], _log_int(rng, 1, case["capacity"])])
            case["window"] = {0: 0, 1: _log_int(rng, 1, case["capacity"]), 2: _log_int(rng, 128, 8192)}[case["window"]]
            return case
        case["backward"] = rng.random() < 0.6
        Sk = _log_int(rng, 1, 16384)
        case["window"] = {0: 0, 1: _log_int(rng, 1, Sk), 2: _log_int(rng, 64, 4096)}[case["window"]]
        case["Sk"] = Sk
        case["Sq"] = Sk if case["backward"] or rng.random() < 0.5 else _log_int(rng, 1, Sk)
        case["B"] = 1
        room = (1 << 40) / work(case)["flops"]          # of the largest listed case
        if room < 1:
            case["Hq"] = case["Hkv"] = 1
        case["B"] = _log_int(rng, 1, max(1, min(8, int(room))))
        return case
    if op == "layernorm":
        times = rng.choice([1, 8])
        H = rng.choice([rng.choice([64, 128]) * rng.choice([1, 2, 4, 8, 16, 20, 32, 40, 64]),
                        (_log_int(rng, 64 // times, 16384 // times - 1) | 1) * times])
        return {"op": op, "M": _log_int(rng, 1, max(1, min(32768, (1 << 26) // H))), "H": H,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "backward": rng.random() < 0.5}
    case = {"op": op, "sizes": rng.choice(["layers", "ragged"]), "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"]),
            "bits": rng.choice([8, 32])}
    if case["sizes"] == "layers":
        case["width"] = 8 * (_log_int(rng, 8, 256) | 1)
        case["count"] = _log_int(rng, 1, max(1, min(48, (1 << 27) // (12 * case["width"] ** 2))))
    else:
        case["count"] = _log_int(rng, 1, 600)
        case["width"] = _log_int(rng, 1, 100000)
    return case


def _ceil(a, b):
    return -(-a // b)


def _sizes(case):
    """Elements of each tensor of an adamw case."""
    w, n = case["width"], case["count"]
    if case["sizes"] == "layers":
        return [3 * w * w, 3 * w, w * w, w, w, 4 * w * w, 4 * w * w, w, w] * n
    return [1 + (i * 7919 * 31 + w) % (2 * w) for i in range(n)]       # 1 to twice the width, most of them odd


def _places(case):
    """Where each tensor begins in a flat buffer, at multiples of 512 elements, and the buffer's length."""
    at = [0]
    for n in _sizes(case):
        at.append(_ceil(at[-1] + n, 512) * 512)
    return at[:-1], at[-1]


def _pairs(case):
    """Visible pairs of a query and a key, of one head of one sequence."""
    Sq, Sk, window, sinks = case["Sq"], case["Sk"], case["window"] or case["Sk"], case["sinks"]
    p = torch.arange(max(0, Sk - Sq), Sk)
    low = (p - window + 1).clamp_min(0)
    return int((p + 1 - low + torch.minimum(low, torch.tensor(sinks))).sum())


def _lengths(case):
    """Tokens of each sequence of a decode case: from the shortest to the whole cache, spread over the logarithm."""
    B, low, high = case["B"], case["shortest"], case["capacity"]
    return [round(math.exp(math.log(low) + (math.log(high) - math.log(low)) * (b + 1) / B)) for b in range(B)]


def work(case):
    op = case["op"]
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if op == "attention":
        q, kv = case["B"] * case["Hq"] * case["Sq"] * case["d"], case["B"] * case["Hkv"] * case["Sk"] * case["d"]
        pairs = case["B"] * case["Hq"] * _pairs(case)
        if not case["backward"]:                       # q, k, v, o
            return {"bytes": size * (2 * q + 2 * kv), "flops": 4 * pairs * case["d"]}
        return {"bytes": size * (4 * q + 4 * kv), "flops": 14 * pairs * case["d"]}     # and dO, dQ, dK, dV
    if op == "decode":
        window = case["window"] or case["capacity"]
        seen = sum(n if n <= window else window + min(case["sinks"], n - window) for n in _lengths(case))
        return {"bytes": size * (2 * seen * case["Hkv"] + 2 * case["B"] * case["Hq"]) * case["d"] + 4 * case["B"],
                "flops": 4 * seen * case["Hq"] * case["d"]}
    if op == "layernorm":
        M, H = case["M"], case["H"]
        if not case["backward"]:      # x, residual, h; 8-bit values and scales; mean and rstd; weight and bias
            return {"bytes": M * H * (3 * size + 1) + M * _ceil(H, BLOCK) + 8 * M + 2 * H * size, "flops": 9 * M * H}
        # dy, h, the residual stream's gradient, dx; mean and rstd; weight, its gradient and the bias's
        return {"bytes": M * H * 4 * size + 8 * M + H * (size + 8), "flops": 15 * M * H}
    n = sum(_sizes(case))
    state = 8 if case["bits"] == 32 else 2            # both states; in 8 bits a scale for 128 values of each
    scales = 0 if case["bits"] == 32 else 2 * sum(_ceil(x, BLOCK) for x in _sizes(case))
    return {"bytes": n * (3 * size + 2 * state) + 2 * scales, "flops": 16 * n}


# ---- plain forms, in 32 bits -------------------------------------------------------------------------

def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within what e8m0 holds; 0 for a block of zeros."""
    m, e = torch.frexp(amax / E4M3_MAX)            # m in [0.5, 1); the quotient of m = 0.5 is a power of two
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(torch.ldexp(torch.full_like(amax, E4M3_MAX), e) < amax, e + 1, e)   # the quotient was rounded
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _row_exponents(x):
    """(exponent of each 128 values of a row, the same spread over the values)."""
    M, N = x.shape
    n = _ceil(N, BLOCK)
    e = _exponent(torch.nn.functional.pad(x.abs(), (0, n * BLOCK - N)).view(M, n, BLOCK).amax(dim=2))
    return e, e.repeat_interleave(BLOCK, 1)[:, :N]


def _scales(e):
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_attention(s):
    """Rows of queries in pieces, against the keys that any of them sees."""
    q, k, v, do = (s[n].float() if n in s else None for n in ("q", "k", "v", "do"))
    B, Sq, Hq, d = q.shape
    Sk, Hkv = k.shape[1:3]
    window, sinks, scale = s["window"] or Sk, s["sinks"], d ** -0.5
    q = q.view(B, Sq, Hkv, Hq // Hkv, d)
    out = torch.empty_like(q)
    if do is not None:
        do = do.view(q.shape)
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = max(1, min(1024, (1 << 28) // (B * Hq * min(Sk, window + sinks + 1024))))
    for i0 in range(0, Sq, rows):
        i1 = min(Sq, i0 + rows)
        p = torch.arange(i0 + Sk - Sq, i1 + Sk - Sq, device=q.device)
        low = max(0, i0 + Sk - Sq - window + 1)
        j = torch.cat([torch.arange(0, min(sinks, low), device=q.device),
                       torch.arange(low, i1 + Sk - Sq, device=q.device)])
        sees = (j <= p[:, None]) & ((j > p[:, None] - window) | (j < sinks))
        qi, kj, vj = q[:, i0:i1], k[:, j], v[:, j]
        a = torch.einsum("bihgd,bjhd->bhgij", qi, kj) * scale
        a = a.masked_fill(~sees, -math.inf)
        a = torch.exp(a - a.amax(dim=-1, keepdim=True))
        a = a / a.sum(dim=-1, keepdim=True)
        out[:, i0:i1] = torch.einsum("bhgij,bjhd->bihgd", a, vj)
        if do is None:
            continue
        di = do[:, i0:i1]
        dv.index_add_(1, j, torch.einsum("bhgij,bihgd->bjhd", a, di))
        da = torch.einsum("bihgd,bjhd->bhgij", di, vj)
        da = a * (da - (a * da).sum(dim=-1, keepdim=True)) * scale
        dq[:, i0:i1] = torch.einsum("bhgij,bjhd->bihgd", da, kj)
        dk.index_add_(1, j, torch.einsum("bhgij,bihgd->bjhd", da, qi))
    t = s["q"].dtype
    got = {"o": out.view(B, Sq, Hq, d).to(t)}
    if do is not None:
        got.update(dq=dq.view(B, Sq, Hq, d).to(t), dk=dk.to(t), dv=dv.to(t))
    return got


def _plain_decode(s):
    q, n = s["q"].float(), s["lengths"].long()[:, None]
    B, Hq, d = q.shape
    capacity, Hkv = s["k"].shape[1:3]
    j = torch.arange(capacity, device=q.device).expand(B, capacity)
    if s["window"] and s["window"] + s["sinks"] < capacity:       # the first tokens, then the window
        first = j[:, :s["sinks"]]
        last = n - s["window"] + j[:, :s["window"]]
        sees = torch.cat([first < n - s["window"], last >= 0], dim=1)
        j = torch.cat([first, last], dim=1).clamp_min(0)
    else:
        sees = j < n
        if s["window"]:
            sees = sees & ((j >= n - s["window"]) | (j < s["sinks"]))
    b = torch.arange(B, device=q.device)[:, None]
    k, v = s["k"][b, j].float(), s["v"][b, j].float()
    a = torch.einsum("bhgd,bjhd->bhgj", q.view(B, Hkv, Hq // Hkv, d), k) * d ** -0.5
    a = a.masked_fill(~sees[:, None, None], -math.inf)
    a = torch.exp(a - a.amax(dim=-1, keepdim=True))
    a = a / a.sum(dim=-1, keepdim=True)
    return {"o": torch.einsum("bhgj,bjhd->bhgd", a, v).reshape(B, Hq, d).to(s["q"].dtype)}


def _plain_layernorm(s):
    if s["backward"]:
        dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        n = (h - s["mean"][:, None]) * rstd
        g = dy * s["weight"].float()
        dx = (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True)) * rstd + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * n).sum(dim=0), "dbias": dy.sum(dim=0)}
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = h.float()
    mean = f.mean(dim=1)
    f = f - mean[:, None]
    rstd = torch.rsqrt(f.square().mean(dim=1) + EPS)
    y = f * rstd[:, None] * s["weight"].float() + s["bias"].float()
    e, each = _row_exponents(y)
    return {"h": h, "q": torch.ldexp(y, -each).to(torch.float8_e4m3fn), "scales": _scales(e), "mean": mean, "rstd": rstd}


def _mix(x):
    """A 32-bit number from another (held in 64 bits), as good as random."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_bits(count, tensor, device):
    """32 bits for each element, from the seed, the step, the tensor's number and the element's."""
    key = _mix(_mix(_mix(ADAM["seed"]) ^ ADAM["step"]) ^ tensor)
    i = torch.arange(count, device=device)
    return _mix((i * 0x9E3779B9 + key) & 0xFFFFFFFF)


def _plain_state(x, r):
    """x [1, n] to 8 bits: rounded up or down to the grid by the 16 bits r, with the fraction as probability."""
    e, each = _row_exponents(x)
    y = torch.ldexp(x, -each)
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp_min(-5) - 4)
    y = torch.copysign(torch.floor(y.abs() / step + (r + 0.5) / 65536) * step, y)
    return y, e


def _plain_adamw(s):
    a = ADAM
    c1, c2 = 1 - a["beta1"] ** a["step"], 1 - a["beta2"] ** a["step"]
    for t, (p, g, m, v) in enumerate(zip(s["params"], s["grads"], s["m"], s["v"])):
        f, n = g.float(), p.numel()
        m8, v8 = s["m_scales"][t], s["v_scales"][t]
        mf, vf = m, v
        if m8 is not None:
            mf, vf = (torch.ldexp(q.float(), (e.view(torch.uint8).int() - 127).repeat_interleave(BLOCK)[:n])
                      for q, e in ((m, m8), (v, v8)))
            vf = vf.square()
        mf = a["beta1"] * mf + (1 - a["beta1"]) * f
        vf = a["beta2"] * vf + (1 - a["beta2"]) * f.square()
        w = p.float() * (1 - a["lr"] * a["weight_decay"])
        p.copy_(w - a["lr"] / c1 * mf / (vf.sqrt() / math.sqrt(c2) + a["eps"]))
        if m8 is None:
            m.copy_(mf)
            v.copy_(vf)
            continue
        r = _random_bits(n, t, p.device)
        q, e = _plain_state(mf[None], r & 0xFFFF)
        m.copy_(q[0])
        m8.copy_(_scales(e)[0])
        root = vf.sqrt()[None]
        q, e = _plain_state(root, r >> 16)
        v.copy_(torch.where((q == 0) & (root > 0), torch.full_like(q, 2.0 ** -9), q)[0])    # not zero stays so
        v8.copy_(_scales(e)[0])
    return s["flat"]


# ---- this package ------------------------------------------------------------------------------------

def _own(s):
    op = s["op"]
    if op == "attention":
        from sequence_re_layout_gb300 import attention, autograd
        mask = {"window": s["window"] or None, "sinks": s["sinks"]}
        if "do" not in s:
            return {"o": attention.forward(s["q"], s["k"], s["v"], **mask)[0]}
        leaves = [s[n].detach().requires_grad_() for n in ("q", "k", "v")]
        o = autograd.attention(*leaves, **mask)
        dq, dk, dv = torch.autograd.grad(o, leaves, s["do"])
        return {"o": o.detach(), "dq": dq, "dk": dk, "dv": dv}
    if op == "decode":
        from sequence_re_layout_gb300 import attention
        return {"o": attention.decode(s["q"], s["k"], s["v"], s["lengths"], window=s["window"] or None,
                                      sinks=s["sinks"])}
    if op == "layernorm":
        from sequence_re_layout_gb300 import fp8
        if s["backward"]:
            dx, dweight, dbias = fp8.layernorm_backward(s["dy"], s["h"], s["mean"], s["rstd"], s["weight"], dh=s["dh"])
            return {"dx": dx, "dweight": dweight, "dbias": dbias}
        y, h, mean, rstd = fp8.layernorm(s["x"], s["weight"], s["bias"], residual=s["residual"], eps=EPS)
        return {"h": h, "q": y.data, "scales": y.scales, "mean": mean, "rstd": rstd}
    from sequence_re_layout_gb300 import fp8, optim
    m, v = s["m"], s["v"]
    if s["m_scales"][0] is not None:
        m = [fp8.Quantized(q[None], e[None]) for q, e in zip(m, s["m_scales"])]
        v = [fp8.Quantized(q[None], e[None]) for q, e in zip(v, s["v_scales"])]
    a = ADAM
    optim.adamw(s["params"], s["grads"], m, v, step=a["step"], lr=a["lr"], betas=(a["beta1"], a["beta2"]),
                eps=a["eps"], weight_decay=a["weight_decay"], seed=a["seed"])
    return s["flat"]


def _plain(s):
    return {"attention": _plain_attention, "decode": _plain_decode, "layernorm": _plain_layernorm,
            "adamw": _plain_adamw}[s["op"]](s)


def run(state):
    return _own(state) if own else _plain(state)


# ---- inputs ------------------------------------------------------------------------------------------

def _activations(M, N, gen, dtype):
    """Values of a residual stream: normal, with a few channels much larger than the rest."""
    x = torch.randn(M, N, generator=gen, device="cuda")
    channel = torch.exp(torch.randn(N, generator=gen, device="cuda"))
    return (x * channel).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    if op == "attention":
        B, Sq, Sk, Hq, Hkv, d = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hkv", "d"))
        s = {"op": op, "window": case["window"], "sinks": case["sinks"], "q": normal(B, Sq, Hq, d),
             "k": normal(B, Sk, Hkv, d), "v": normal(B, Sk, Hkv, d)}
        if case["backward"]:
            s["do"] = normal(B, Sq, Hq, d)
        return s
    if op == "decode":
        B, n, Hq, Hkv, d = (case[n] for n in ("B", "capacity", "Hq", "Hkv", "d"))
        return {"op": op, "window": case["window"], "sinks": case["sinks"], "q": normal(B, Hq, d),
                "k": normal(B, n, Hkv, d), "v": normal(B, n, Hkv, d),
                "lengths": torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")}
    if op == "layernorm":
        M, H = case["M"], case["H"]
        s = {"op": op, "backward": case["backward"],
             "weight": (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)}
        if not case["backward"]:
            s.update(x=normal(M, H), residual=_activations(M, H, gen, dtype), bias=0.1 * normal(H))
            return s
        h = _activations(M, H, gen, dtype)
        mean = h.float().mean(dim=1)
        rstd = torch.rsqrt((h.float() - mean[:, None]).square().mean(dim=1) + EPS)
        s.update(h=h, mean=mean, rstd=rstd, dy=normal(M, H), dh=normal(M, H))
        return s
    # the tensors are pieces of flat buffers, as a program that reduces its gradients in buckets has them
    at, total = _places(case)
    inside = torch.zeros(total + 1, dtype=torch.int32, device="cuda")
    begin = torch.tensor(at, device="cuda")
    inside[begin] += 1
    inside[begin + torch.tensor(_sizes(case), device="cuda")] -= 1
    inside = inside.cumsum(0)[:total]
    # gradients of very different sizes from one part of a tensor to the next
    size = torch.exp(2 * torch.randn(total // 64, generator=gen, device="cuda") - 7).repeat_interleave(64) * inside
    g, m, root = (torch.randn(total, generator=gen, device="cuda") * size for _ in range(3))
    flat = {"p": (0.02 * inside * torch.randn(total, generator=gen, device="cuda")).to(dtype), "g": g.to(dtype)}
    m, root = 0.3 * m, 0.1 * (root.abs() + size)
    if case["bits"] == 32:
        flat.update(m=m, v=root.square())
    else:
        (me, each), (ve, each_v) = _row_exponents(m[None]), _row_exponents(root[None])
        root = torch.ldexp(root[None], -each_v).clamp_min(2.0 ** -9) * inside
        flat.update(m=torch.ldexp(m[None], -each).to(torch.float8_e4m3fn)[0], m_scales=_scales(me)[0],
                    v=root.to(torch.float8_e4m3fn)[0], v_scales=_scales(ve)[0])
    s = {"op": op, "flat": {n: x for n, x in flat.items() if n != "g"}}
    for name, key in (("params", "p"), ("grads", "g"), ("m", "m"), ("v", "v")):
        s[name] = [flat[key][i:i + n] for i, n in zip(at, _sizes(case))]
    for key in ("m_scales", "v_scales"):
        s[key] = [flat[key][i // BLOCK:i // BLOCK + _ceil(n, BLOCK)] if key in flat else None
                  for i, n in zip(at, _sizes(case))]
    return s


# ---- 64 bits, from the definitions -------------------------------------------------------------------

def _exact_attention(case, s):
    """Head by head: every pair of a piece of queries and all keys up to them."""
    B, Sq, Sk, Hq, Hkv = (case[n] for n in ("B", "Sq", "Sk", "Hq", "Hkv"))
    group, scale = Hq // Hkv, 1 / math.sqrt(case["d"])
    got = {"o": torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")}
    if case["backward"]:
        got.update({"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")})
    piece = 2048
    for b in range(B):
        for head in range(Hq):
            k, v = (s[n][b, :, head // group].double() for n in ("k", "v"))
            for begin in range(0, Sq, piece):
                end = min(Sq, begin + piece)
                at = torch.arange(begin, end, device="cuda").unsqueeze(1) + (Sk - Sq)
                first = max(0, begin + Sk - Sq - (case["window"] or Sk) + 1)
                first = 0 if first <= case["sinks"] else first
                parts = [(first, end + Sk - Sq)] if first == 0 else [(0, case["sinks"]), (first, end + Sk - Sq)]
                key = torch.cat([torch.arange(x, y, device="cuda") for x, y in parts if y > x])
                hidden = (key > at) | ((at - key >= (case["window"] or Sk)) & (key >= case["sinks"]))
                q, kk, vv = s["q"][b, begin:end, head].double(), k[key], v[key]
                score = (q @ kk.T).mul_(scale).masked_fill_(hidden, -math.inf)
                prob = torch.exp(score - torch.logsumexp(score, dim=1, keepdim=True))
                got["o"][b, begin:end, head] = prob @ vv
                if case["backward"]:
                    do = s["do"][b, begin:end, head].double()
                    got["dv"][b, :, head // group].index_add_(0, key, prob.T @ do)
                    delta = (do * (prob @ vv)).sum(dim=1, keepdim=True)
                    ds = prob * (do @ vv.T - delta)
                    got["dq"][b, begin:end, head] = scale * (ds @ kk)
                    got["dk"][b, :, head // group].index_add_(0, key, scale * (ds.T @ q))
    return got


def _exact_decode(case, s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["Hq"] // case["Hkv"]
    for b, n in enumerate(_lengths(case)):
        first = max(0, n - (case["window"] or n))
        key = list(range(min(first, case["sinks"]))) + list(range(first, n))
        key = torch.tensor(key, device="cuda")
        k, v = s["k"][b, key].double(), s["v"][b, key].double()              # [n, Hkv, d]
        q = s["q"][b].double().unflatten(0, (case["Hkv"], group))
        prob = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(case["d"]), dim=2)
        out[b] = torch.einsum("hgn,nhd->hgd", prob, v).flatten(0, 1)
    return {"o": out}


def _exact_scale(x):
    """e for each 128 values of a row, from the definition, and for each value."""
    blocks = [x[:, c:c + BLOCK].abs().amax(dim=1) for c in range(0, x.shape[1], BLOCK)] if x.shape[0] > 1 else \
        [torch.nn.functional.pad(x[0].abs(), (0, -x.shape[1] % BLOCK)).view(-1, BLOCK).amax(dim=1)]
    amax = torch.stack(blocks, dim=1) if x.shape[0] > 1 else blocks[0][None]
    e = torch.ceil(torch.log2(amax / E4M3_MAX))
    e = torch.where(E4M3_MAX * torch.exp2(e - 1) >= amax, e - 1, e)     # log2 next to a whole number
    e = torch.where(E4M3_MAX * torch.exp2(e) < amax, e + 1, e)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    return e, e[:, torch.arange(x.shape[1], device=x.device) // BLOCK]


def _grid_step(y):
    """Distance of two neighbouring e4m3 values at |y|: 3 bits; subnormals below 2^-6."""
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)


def _exact_layernorm(case, s):
    w = s["weight"].double()
    if case["backward"]:
        # d/dh of (h - mean) r w with the mean and r as they were saved, plus the residual stream's gradient
        dy, r, H = s["dy"].double(), s["rstd"].double().unsqueeze(1), case["H"]
        c = s["h"].double() - s["mean"].double().unsqueeze(1)
        z = dy * w
        dx = r * z - r / H * z.sum(1, keepdim=True) - c * r.pow(3) / H * (z * c).sum(1, keepdim=True)
        return {"dx": dx + s["dh"].double(), "dweight": (dy * c * r).sum(0), "dbias": dy.sum(0)}
    h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    mean = h.sum(dim=1) / h.shape[1]
    rstd = ((h - mean.unsqueeze(1)).pow(2).sum(dim=1) / h.shape[1] + EPS).pow(-0.5)
    y = (h - mean.unsqueeze(1)) * rstd.unsqueeze(1) * w + s["bias"].double()
    e, each = _exact_scale(y)
    y = y * torch.exp2(-each)
    step = _grid_step(y)
    return {"h": h, "q": torch.round(y / step) * step, "scales": torch.exp2(e), "mean": mean, "rstd": rstd}


def _exact_hash(x):
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
        x = ((x ^ (x >> shift)) * factor) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _exact_adamw(case, s):
    a, eight = ADAM, case["bits"] == 8
    got = {}
    for name, x in s["flat"].items():
        got[name] = torch.exp2(x.view(torch.uint8).double() - 127) if "scales" in name else x.float().double()
    t = a["step"]
    for number, (n, place) in enumerate(zip(_sizes(case), _places(case)[0])):
        here, blocks = slice(place, place + n), slice(place // BLOCK, place // BLOCK + _ceil(n, BLOCK))
        g, p, m, v = s["grads"][number].double(), got["p"][here], got["m"][here], got["v"][here]
        if eight:
            block = torch.arange(n, device="cuda") // BLOCK
            m, v = m * got["m_scales"][blocks][block], (v * got["v_scales"][blocks][block]).pow(2)
        m = m + (1 - a["beta1"]) * (g - m)
        v = v + (1 - a["beta2"]) * (g * g - v)
        up = (m / (1 - a["beta1"] ** t)) / ((v / (1 - a["beta2"] ** t)).sqrt() + a["eps"])
        got["p"][here] = p - a["lr"] * (up + a["weight_decay"] * p)
        if not eight:
            got["m"][here], got["v"][here] = m, v
            continue
        key = _exact_hash(_exact_hash(_exact_hash(a["seed"]) ^ t) ^ number)
        bits = _exact_hash((torch.arange(n, device="cuda") * 0x9E3779B9 + key) & 0xFFFFFFFF)
        for name, x, r in (("m", m, bits % 65536), ("v", v.sqrt(), bits // 65536)):
            e, each = _exact_scale(x[None])
            y = x[None] * torch.exp2(-each)
            step = _grid_step(y)
            low = torch.floor(y.abs() / step)
            up = (y.abs() / step - low) + (r.double() + 0.5) / 65536 >= 1
            q = torch.sign(y) * (low + up) * step
            got[name][here] = (q if name == "m" else torch.where((y > 0) & (q == 0), 2.0 ** -9, q))[0]
            got[name + "_scales"][blocks] = torch.exp2(e)[0]
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        if work(case)["flops"] * case["B"] * case["Hq"] > 1 << 47:      # many heads, much work: too long in 64 bits
            return None
        return _exact_attention(case, s)
    return {"decode": _exact_decode, "layernorm": _exact_layernorm, "adamw": _exact_adamw}[case["op"]](case, s)
