"""Plain 64-bit forms of the 8-bit operators, from their definitions, on the CPU
(numpy only; shares no code with the CUDA path).

An 8-bit matrix is a pair (values, exponents): values on the e4m3 grid as
float64, and one exponent e for each block, the element standing for
value * 2^e."""
import numpy as np

BLOCK = 128
E4M3_MAX = 448.0


def least_exponent(amax):
    """The least e >= -127 with amax <= 448 * 2^e, by trying; 0 for zero."""
    if amax == 0:
        return 0
    e = -127
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


def round_e4m3(v):
    """Nearest e4m3 value, ties to even: 3 mantissa bits down to 2^-6, then
    steps of 2^-9."""
    v = np.asarray(v, dtype=np.float64)
    exponent = np.frexp(np.where(np.isfinite(v), v, 0.0))[1] - 1        # |v| in [2^x, 2^(x+1))
    step = 2.0 ** (np.maximum(exponent, -6) - 3)
    return np.where(np.isfinite(v), np.round(np.where(np.isfinite(v), v, 0.0) / step) * step, np.nan)


def quantize(x, block_rows):
    """(values, exponents) of a float64 matrix: the scale comes from the largest
    finite magnitude, infinities and NaN become NaN."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    er, ec = -(-rows // block_rows), -(-cols // BLOCK)
    values, exps = np.zeros_like(x), np.zeros((er, ec), dtype=np.int64)
    for i in range(er):
        for j in range(ec):
            at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            b = x[at]
            finite = np.abs(b[np.isfinite(b)])
            exps[i, j] = least_exponent(finite.max() if finite.size else 0.0)
            values[at] = round_e4m3(b * 2.0 ** -float(exps[i, j]))
    return values, exps


def dequantize(values, exps, block_rows):
    rows, cols = values.shape
    r, c = np.arange(rows) // block_rows, np.arange(cols) // BLOCK
    return values * 2.0 ** exps[r][:, c].astype(np.float64)


def norm(h, weight, eps):
    """(y, rstd) of float64 rows."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * weight, rstd


def norm_backward(dy, h, rstd, weight, dh):
    """(dx, dweight): the derivative of norm() times dy, plus dh."""
    g, n = dy * weight, h * rstd[:, None]
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return dx + (0 if dh is None else dh), (dy * n).sum(axis=0)
