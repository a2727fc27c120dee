"""Plain 64-bit forms of the layer norm, the attention and the optimiser's step, from
their definitions, on the CPU (numpy only; shares no code with the CUDA path), and
bounds of what the kernels' roundings can make of them.

A rounding to a type t is off by at most u(t) = finfo(t).eps / 2 of the value, and by
TINY near zero (fp16's last step is 2^-24).  The tensor cores truncate where they
add: a sum of n products is off by at most n * 2^-23 of its sum of magnitudes."""
import numpy as np

F32 = 2.0 ** -24
TINY = 2.0 ** -25


def layernorm(h, weight, bias, eps):
    """(y, mean, rstd) of float64 rows."""
    mean = h.mean(axis=1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    return c * rstd[:, None] * weight + (0 if bias is None else bias), mean, rstd


def layernorm_backward(dy, h, mean, rstd, weight, dh):
    """(dx, dweight, dbias): the derivative of layernorm() times dy, plus dh."""
    g, n = dy * weight, (h - mean[:, None]) * rstd[:, None]
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - n * (g * n).mean(axis=1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * n).sum(axis=0), dy.sum(axis=0)


def visible(sq, sk, window, sinks):
    """[sq, sk]: whether a query sees a key."""
    p, j = np.arange(sq)[:, None] + sk - sq, np.arange(sk)[None]
    near = True if window is None else j > p - window
    return (j <= p) & (near | (j < sinks))


class Attention:
    """One sequence's attention in 64 bits: q [sq, hq, d], k, v [sk, hkv, d], and a
    bound for each result of a kernel whose P and dS are rounded to a type of
    half-step u before their products.

    A score is off by es = |scale| (d + 8) 2^-23 sum |q||k| and a few roundings of
    itself; P by that twice (its own, and the row's sum's), the exponential's 2^-21
    and n 2^-24 of the sum.  What is added over n terms is off by (n + 16) 2^-23 of its
    magnitudes."""

    def __init__(self, q, k, v, window, sinks, scale, u):
        self.q, self.k, self.v, self.scale, self.u = q, k, v, scale, u
        sq, hq, d = q.shape
        sk, hkv, _ = k.shape
        self.group, self.sees = hq // hkv, visible(sq, sk, window, sinks)
        self.n = max(sq, sk)
        self.add = (self.n + 16) * 2.0 ** -23
        self.o, self.lse = np.zeros(q.shape), np.full((hq, sq), -np.inf)
        self.o_bound, self.lse_bound = np.zeros(q.shape), np.zeros((hq, sq))
        self.p, self.ep = {}, {}
        for h in range(hq):
            kh, vh = k[:, h // self.group], v[:, h // self.group]
            with np.errstate(invalid="ignore"):
                s = np.where(self.sees, scale * (q[:, h] @ kh.T), -np.inf)
            es = abs(scale) * (d + 8) * 2.0 ** -23 * (np.abs(q[:, h]) @ np.abs(kh).T) + 2.0 ** -22 * np.abs(
                np.where(self.sees, s, 0))
            es = np.where(self.sees, es, 0)
            m = np.where(self.sees.any(1), s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - m[:, None])
            l = e.sum(1)
            p = e / np.where(l > 0, l, 1)[:, None]
            # relative error of P: its score's, the sum's, the exponential's
            worst = es.max(1, initial=0.0)[:, None]
            ep = p * (np.expm1(2 * worst) + 2.0 ** -20 + self.n * F32 * 2)
            some = l > 0
            self.lse[h, some] = m[some] + np.log(l[some])
            self.lse_bound[h] = worst[:, 0] + 2.0 ** -20 + self.n * F32 * 2 + 2.0 ** -22 * np.abs(
                np.where(some, self.lse[h], 0))
            self.p[h], self.ep[h] = p, ep
            self.o[:, h] = p @ vh
            # P before its division is at least TINY off where it is small (its largest is
            # 1 or more, so that divided by the row's sum it is no worse)
            rounding = p * u + np.where(self.sees, 2 * TINY, 0)
            self.o_bound[:, h] = (ep + rounding) @ np.abs(vh) + self.add * (p @ np.abs(vh)) + \
                u * np.abs(self.o[:, h]) + TINY

    def backward(self, do, o_rounding):
        """dq, dk, dv and their bounds; o_rounding is the error of the o that D is made of."""
        got = {n: np.zeros(x.shape) for n, x in (("dq", self.q), ("dk", self.k), ("dv", self.v))}
        bound = {n: np.zeros(x.shape) for n, x in (("dq", self.q), ("dk", self.k), ("dv", self.v))}
        d, u, scale = self.q.shape[2], self.u, self.scale
        for h in range(self.q.shape[1]):
            kv = h // self.group
            p, ep, g = self.p[h], self.ep[h], do[:, h]
            dp = np.where(self.sees, g @ self.v[:, kv].T, 0)
            edp = np.where(self.sees, (d + 8) * 2.0 ** -23 * (np.abs(g) @ np.abs(self.v[:, kv]).T), 0)
            delta = (g * self.o[:, h]).sum(1)[:, None]
            ed = (np.abs(g) * (o_rounding[:, h] + (d + 8) * F32 * np.abs(self.o[:, h]))).sum(1)[:, None]
            ds = p * (dp - delta)
            eds = ep * (np.abs(dp) + np.abs(delta)) + (p + ep) * (edp + ed + 2 * F32 * (np.abs(dp) + np.abs(delta)))
            eds = np.where(self.sees, eds + u * (np.abs(ds) + eds) + TINY, 0)
            erp = np.where(self.sees, ep + u * (p + ep) + TINY, 0)
            for name, a, ea, b, at, c in (("dv", p.T, erp.T, g, kv, 1.0), ("dk", ds.T, eds.T, self.q[:, h], kv, scale),
                                          ("dq", ds, eds, self.k[:, kv], h, scale)):
                got[name][:, at] += c * (a @ b)
                bound[name][:, at] += abs(c) * (ea @ np.abs(b) + self.add * self.group * (np.abs(a) @ np.abs(b)))
        for name in got:
            bound[name] += u * np.abs(got[name]) + TINY
        return got, bound


# ---- the optimiser's step ---------------------------------------------------------

M32 = 0xFFFFFFFF


def mix(x):
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x6A09E667) & np.uint64(M32)
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0xBB67AE85) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random_bits(n, seed, step, tensor):
    """(low 16 bits, high 16 bits) for each of n elements."""
    key = mix(mix(mix(seed) ^ np.uint64(step)) ^ np.uint64(tensor))
    bits = mix((np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B9) + key) & np.uint64(M32))
    return bits & np.uint64(0xFFFF), bits >> np.uint64(16)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """(p, m, v) after one step, in 64 bits."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    up = (m / (1 - beta1 ** step)) / (np.sqrt(v) / np.sqrt(1 - beta2 ** step) + eps)
    return p * (1 - lr * weight_decay) - lr * up, m, v


def round_at_random(y, r):
    """(value, how far its decision is from the other one, in steps): y within 448 to the e4m3 grid."""
    step = 2.0 ** (np.maximum(np.frexp(np.abs(y))[1] - 1, -6) - 3)
    k = np.floor(np.abs(y) / step)
    t = np.abs(y) / step - k + (r + 0.5) / 65536
    return np.copysign((k + (t >= 1)) * step, y), np.abs(t - 1)


def gradients_in_units(a, do, o_rounding, p_unit, q_unit, k_unit):
    """(dq, dk, dv) of an Attention and their bounds, where P of dv is rounded as p_unit times
    it, dS of dq as q_unit [hq, sq] times it and dS of dk as k_unit times it: fp16's last step,
    TINY, is that much smaller.  The rest as in Attention.backward."""
    got = {n: np.zeros(x.shape) for n, x in (("dq", a.q), ("dk", a.k), ("dv", a.v))}
    bound = {n: np.zeros(x.shape) for n, x in got.items()}
    d, u = a.q.shape[2], a.u
    for h in range(a.q.shape[1]):
        kv, p, ep, g = h // a.group, a.p[h], a.ep[h], do[:, h]
        dp = np.where(a.sees, g @ a.v[:, kv].T, 0)
        size = np.where(a.sees, np.abs(g) @ np.abs(a.v[:, kv]).T, 0)
        delta = (g * a.o[:, h]).sum(1)[:, None]
        ed = (np.abs(g) * (o_rounding[:, h] + (d + 8) * F32 * np.abs(a.o[:, h]))).sum(1)[:, None]
        ds = p * (dp - delta)
        e = ep * (np.abs(dp) + np.abs(delta)) + (p + ep) * ((d + 8) * 2.0 ** -23 * size + ed + 2 * F32 * (np.abs(dp) + np.abs(delta)))
        rounded = lambda x, ex, unit: np.where(a.sees, ex + u * (np.abs(x) + ex) + TINY / unit, 0)       # noqa: E731
        for name, x, ex, y, at, c in (("dv", p.T, rounded(p, ep, p_unit).T, g, kv, 1.0),
                                      ("dk", ds.T, rounded(ds, e, k_unit).T, a.q[:, h], kv, a.scale),
                                      ("dq", ds, rounded(ds, e, q_unit[h][:, None]), a.k[:, kv], h, a.scale)):
            got[name][:, at] += c * (x @ y)
            bound[name][:, at] += abs(c) * (ex @ np.abs(y) + a.add * a.group * (np.abs(x) @ np.abs(y)))
    for name in got:
        bound[name] += u * np.abs(got[name]) + TINY
    return got, bound
