"""The operators that stand on both sides of the re-layout in a transformer layer, as measurable cases.

A sequence-parallel attention layer norms the residual stream, projects it to Q, K and V, re-lays the
heads out, attends, re-lays back and projects again.  The operators here are those of the projections
in 8-bit floating point:

  norm           residual addition and root-mean-square norm, output in 8 bits with a scale for each
                 128 values of a row
  norm_backward  its gradient for the residual stream and the norm's weight
  quantize       a 16- or 32-bit matrix to 8 bits, with a scale for each 128 values of a row or each
                 block of 128 x 128, and the same for its transpose where a gradient's product needs it
  matmul         the product of two matrices held that way: A[M, K] times B[N, K] transposed

8-bit values are e4m3; scales are powers of two (e8m0).  With ``own`` false, ``run`` computes each one
from elementary torch operations in 32 bits; with ``own`` true it calls this package.
"""
import math

import torch

own = False

BLOCK = 128           # values that share a scale
E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token of a hidden size of 16 heads x 128: what counts is latency
        {"name": "norm_token", "op": "norm", "M": 1, "H": 2048, "dtype": "bf16"},
        # two sequences of 16384 tokens through one layer
        {"name": "norm_long", "op": "norm", "M": 32768, "H": 2048, "dtype": "bf16"},
        # a packed batch of odd length over rows that no vector load fits
        {"name": "norm_ragged", "op": "norm", "M": 4099, "H": 5003, "dtype": "fp16"},
        # the same two sequences on the way back, with the residual stream's own gradient joining
        {"name": "norm_backward_long", "op": "norm_backward", "M": 32768, "H": 2048, "dtype": "bf16"},
        # a short fine-tuning batch of odd length
        {"name": "norm_backward_ragged", "op": "norm_backward", "M": 777, "H": 1999, "dtype": "fp16"},
        # the packed Q, K, V gradient (48 heads x 128) for the products with the weight and the input
        {"name": "quantize_gradient", "op": "quantize", "M": 32768, "N": 6144, "dtype": "bf16", "rows": 1,
         "transposed": True},
        # the packed projection's 32-bit master weight, once a step, for both directions
        {"name": "quantize_weight", "op": "quantize", "M": 6144, "N": 2048, "dtype": "fp32", "rows": 128,
         "transposed": True},
        # one decoded token through the packed Q, K, V projection, which has a bias
        {"name": "matmul_token", "op": "matmul", "M": 1, "N": 6144, "K": 2048, "rows_b": 128, "out": "bf16",
         "bias": True},
        # a decode batch through the output projection
        {"name": "matmul_batch", "op": "matmul", "M": 64, "N": 2048, "K": 2048, "rows_b": 128, "out": "bf16",
         "bias": False},
        # odd sizes on every side
        {"name": "matmul_ragged", "op": "matmul", "M": 1021, "N": 2999, "K": 1543, "rows_b": 1, "out": "fp16",
         "bias": True},
        # two sequences of 16384 tokens through the packed Q, K, V projection
        {"name": "matmul_long", "op": "matmul", "M": 32768, "N": 6144, "K": 2048, "rows_b": 128, "out": "bf16",
         "bias": True},
        # the gradient of that projection's weight: the tokens are summed over
        {"name": "matmul_weight_gradient", "op": "matmul", "M": 6144, "N": 2048, "K": 32768, "rows_b": 1,
         "out": "fp32", "bias": False},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _size(rng, low, high):
    """Whole heads, as hidden sizes are; or over the whole range, odd or 8 times an odd number."""
    if rng.random() < 0.5:
        return rng.choice([64, 128]) * rng.choice([1, 2, 4, 8, 16, 20, 32, 40, 64])
    times = rng.choice([1, 8])
    return (_log_int(rng, low // times, high // times - 1) | 1) * times


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "quantize", "matmul", "matmul"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_backward"):
        H = _size(rng, 64, 16384)
        return {"op": op, "M": _log_int(rng, 1, max(1, min(32768, (1 << 26) // H))), "H": H, "dtype": dtype}
    if op == "quantize":
        N = _size(rng, 64, 16384)
        return {"op": op, "M": _log_int(rng, 1, max(1, min(32768, (1 << 27) // N))), "N": N, "dtype": dtype,
                "rows": rng.choice([1, 1, 128]), "transposed": rng.random() < 0.5}
    N, K = _size(rng, 64, 8192), _size(rng, 64, 8192)
    return {"op": op, "M": _log_int(rng, 1, max(1, min(32768, (1 << 38) // (N * K)))), "N": N, "K": K,
            "rows_b": rng.choice([1, 128]), "out": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "bias": rng.random() < 0.5}


def _ceil(a, b):
    return -(-a // b)


def work(case):
    if case["op"] in ("norm", "norm_backward"):
        M, H = case["M"], case["H"]
        size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        if case["op"] == "norm":      # x, residual, new residual; 8-bit values and scales; 1/rms; weight
            return {"bytes": M * H * (3 * size + 1) + M * _ceil(H, BLOCK) + 4 * M + H * size, "flops": 7 * M * H}
        # dy, the normed values, the residual stream's gradient, dx; 1/rms; weight and its gradient
        return {"bytes": M * H * 4 * size + 4 * M + H * (size + 4), "flops": 12 * M * H}
    if case["op"] == "quantize":
        M, N, rows = case["M"], case["N"], case["rows"]
        size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
        out = M * N + _ceil(M, rows) * _ceil(N, BLOCK)
        if case["transposed"]:
            out += M * N + _ceil(N, rows) * _ceil(M, BLOCK)
        return {"bytes": M * N * size + out, "flops": 2 * M * N}
    M, N, K = case["M"], case["N"], case["K"]
    size = torch.finfo(DTYPES[case["out"]]).bits // 8
    scales = _ceil(K, BLOCK) * (M + _ceil(N, case["rows_b"]))
    return {"bytes": K * (M + N) + scales + size * (M * N + (N if case["bias"] else 0)), "flops": 2 * M * N * K}


# ---- plain forms, in 32 bits -------------------------------------------------------------------------

def _block_max(x, rows):
    """Largest magnitude of each block of ``rows`` x 128: [ceil(M / rows), ceil(N / 128)]."""
    M, N = x.shape
    m, n = _ceil(M, rows), _ceil(N, BLOCK)
    x = torch.nn.functional.pad(x.abs(), (0, n * BLOCK - N, 0, m * rows - M))
    return x.view(m, rows, n, BLOCK).amax(dim=(1, 3))


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, within what e8m0 holds; 0 for a block of zeros."""
    m, e = torch.frexp(amax / E4M3_MAX)            # m in [0.5, 1); the quotient of m = 0.5 is a power of two
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(torch.ldexp(torch.full_like(amax, E4M3_MAX), e) < amax, e + 1, e)   # the quotient was rounded
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def _spread(per_block, rows, M, N):
    """One value for each block -> one for each element."""
    return per_block.repeat_interleave(rows, 0)[:M].repeat_interleave(BLOCK, 1)[:, :N]


def _plain_quantize(x, rows):
    e = _exponent(_block_max(x, rows))
    q = torch.ldexp(x, -_spread(e, rows, *x.shape)).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_dequantize(data, scales, rows):
    e = scales.view(torch.uint8).to(torch.int32) - 127
    return torch.ldexp(data.float(), _spread(e, rows, *data.shape))


def _plain(s):
    op = s["op"]
    if op == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        f = h.float()
        rstd = torch.rsqrt(f.square().mean(dim=1) + EPS)
        q, scales = _plain_quantize(f * rstd[:, None] * s["weight"].float(), 1)
        return {"h": h, "q": q, "scales": scales, "rstd": rstd}
    if op == "norm_backward":
        dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
        g = dy * s["weight"].float()
        xhat = h * rstd
        dx = (g - xhat * (g * xhat).mean(dim=1, keepdim=True)) * rstd + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xhat).sum(dim=0)}
    if op == "quantize":
        x = s["x"].float()
        q, scales = _plain_quantize(x, s["rows"])
        if not s["transposed"]:
            return {"q": q, "scales": scales}
        qt, scales_t = _plain_quantize(x.t().contiguous(), s["rows"])
        return {"q": q, "scales": scales, "qt": qt, "scales_t": scales_t}
    c = _plain_dequantize(s["a"], s["a_scales"], 1) @ _plain_dequantize(s["b"], s["b_scales"], s["rows_b"]).t()
    return {"c": (c if s["bias"] is None else c + s["bias"].float()).to(s["out"])}


def _own(s):
    from sequence_re_layout_gb300 import fp8
    op = s["op"]
    if op == "norm":
        y, h, rstd = fp8.rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantized=True)
        return {"h": h, "q": y.data, "scales": y.scales, "rstd": rstd}
    if op == "norm_backward":
        dx, dweight = fp8.rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["weight"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    if op == "quantize":
        if not s["transposed"]:
            q = fp8.quantize(s["x"], block_rows=s["rows"])
            return {"q": q.data, "scales": q.scales}
        q, qt = fp8.quantize(s["x"], block_rows=s["rows"], transposed=True)
        return {"q": q.data, "scales": q.scales, "qt": qt.data, "scales_t": qt.scales}
    a = fp8.Quantized(s["a"], s["a_scales"], 1)
    b = fp8.Quantized(s["b"], s["b_scales"], s["rows_b"])
    return {"c": fp8.matmul(a, b, bias=s["bias"], out_dtype=s["out"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---- inputs ------------------------------------------------------------------------------------------

def _pitched(x, multiple):
    """The same matrix in storage whose rows start at multiples of ``multiple`` bytes (1-byte elements)."""
    M, N = x.shape
    store = torch.zeros(M, _ceil(N, multiple) * multiple, dtype=torch.uint8, device=x.device)
    store[:, :N] = x.view(torch.uint8)
    return store.view(x.dtype)[:, :N]


def _activations(M, N, gen, dtype):
    """Values of a residual stream: normal, with a few channels much larger than the rest."""
    x = torch.randn(M, N, generator=gen, device="cuda")
    channel = torch.exp(torch.randn(N, generator=gen, device="cuda"))
    return (x * channel).to(dtype)


def _quantized(M, K, gen, rows, weight):
    x = torch.randn(M, K, generator=gen, device="cuda") * 0.02 if weight else _activations(M, K, gen, torch.float32)
    q, scales = _plain_quantize(x, rows)
    return _pitched(q, 16), _pitched(scales, 4)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "matmul":
        M, N, K, out = case["M"], case["N"], case["K"], DTYPES[case["out"]]
        a, a_scales = _quantized(M, K, gen, 1, False)
        b, b_scales = _quantized(N, K, gen, case["rows_b"], True)
        bias = torch.randn(N, generator=gen, device="cuda").to(out) if case["bias"] else None
        return {"op": op, "a": a, "a_scales": a_scales, "b": b, "b_scales": b_scales, "rows_b": case["rows_b"],
                "bias": bias, "out": out}
    dtype = DTYPES[case["dtype"]]
    if op == "quantize":
        x = _activations(case["M"], case["N"], gen, dtype)
        return {"op": op, "x": x, "rows": case["rows"], "transposed": case["transposed"]}
    M, H = case["M"], case["H"]
    weight = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
    if op == "norm":
        return {"op": op, "weight": weight, "x": torch.randn(M, H, generator=gen, device="cuda").to(dtype),
                "residual": _activations(M, H, gen, dtype)}
    h = _activations(M, H, gen, dtype)
    rstd = torch.rsqrt(h.float().square().mean(dim=1) + EPS)
    dy, dh = (torch.randn(M, H, generator=gen, device="cuda").to(dtype) for _ in range(2))
    return {"op": op, "weight": weight, "h": h, "rstd": rstd, "dy": dy, "dh": dh}


# ---- 64 bits, from the definitions -------------------------------------------------------------------

def _exact_quantize(x, rows):
    """The e4m3 values nearest to x / 2^e (ties to even), e from the definition, and the scales 2^e."""
    M, N = x.shape
    m, n = _ceil(M, rows), _ceil(N, BLOCK)
    row = torch.arange(M, device=x.device) // rows
    if rows == 1:
        amax = torch.stack([x[:, j * BLOCK:(j + 1) * BLOCK].abs().amax(dim=1) for j in range(n)], dim=1)
    else:
        amax = torch.stack([torch.stack([x[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK].abs().max()
                                         for j in range(n)]) for i in range(m)])
    e = torch.ceil(torch.log2(amax / E4M3_MAX))
    e = torch.where(E4M3_MAX * torch.exp2(e - 1) >= amax, e - 1, e)     # log2 next to a whole number
    e = torch.where(E4M3_MAX * torch.exp2(e) < amax, e + 1, e)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    v = x * torch.exp2(-e)[row][:, torch.arange(N, device=x.device) // BLOCK]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)   # 3 bits; subnormals below 2^-6
    return torch.round(v / step) * step, torch.exp2(e)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "matmul":
        def wide(q, scales, rows):
            v = q.to(torch.float32).double()
            e = scales.view(torch.uint8).double() - 127
            r = torch.arange(v.shape[0], device=v.device) // rows
            c = torch.arange(v.shape[1], device=v.device) // BLOCK
            return v.mul_(torch.exp2(e)[r][:, c])
        c = torch.einsum("mk,nk->mn", wide(s["a"], s["a_scales"], 1), wide(s["b"], s["b_scales"], s["rows_b"]))
        return {"c": c if s["bias"] is None else c.add_(s["bias"].double())}
    if op == "norm":
        h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        rstd = (h.pow(2).sum(dim=1) / h.shape[1] + EPS).pow(-0.5)
        q, scales = _exact_quantize(h * rstd.unsqueeze(1) * s["weight"].double(), 1)
        return {"h": h, "q": q, "scales": scales, "rstd": rstd}
    if op == "norm_backward":
        # d/dh of h * r(h) * w with r = (mean h^2 + eps)^-1/2, r as it was saved, plus the residual stream's gradient
        dy, h, w, r = s["dy"].double(), s["h"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
        dot = (dy * w * h).sum(dim=1, keepdim=True)
        dx = r * w * dy - h * r.pow(3) * dot / h.shape[1] + s["dh"].double()
        return {"dx": dx, "dweight": (dy * h * r).sum(dim=0)}
    if s["x"].numel() > 1 << 28:
        return None
    x = s["x"].double()
    q, scales = _exact_quantize(x, s["rows"])
    if not s["transposed"]:
        return {"q": q, "scales": scales}
    qt, scales_t = _exact_quantize(x.t(), s["rows"])
    return {"q": q, "scales": scales, "qt": qt, "scales_t": scales_t}
