"""8-bit norm and projections on torch tensors, over the C ABI of
``include/basp_fp8.h``: what stands before ``seq2head`` (norm and packed QKV
projection) and after ``head2seq`` (output projection).

    x8, h, rstd = fp8.rmsnorm(x, norm_weight, residual=residual)
    w8 = fp8.quantize(weight, block_rows=128)           # once, or once a step
    qkv = fp8.matmul(x8, w8, bias=bias)                 # -> seq2head_qkv

These functions allocate their outputs and run on the current stream; nothing
synchronises.  They are no operations of autograd: their results carry no gradient
and no tangent (``autograd`` has the differentiable forms), and a tensor given to
write to (``h``, ``out``) may not require a gradient outside of ``torch.no_grad()``.
"""
from __future__ import annotations

import torch

from . import binding

BLOCK = binding.BASP_FP8_BLOCK

_ops = None


def _load():
    """The compiled calls on torch tensors (``csrc/torch_ops.cpp``).  There is
    no fallback: a missing module is an error."""
    global _ops
    try:
        from . import _torch_ops
    except ImportError as e:
        raise ImportError("sequence_re_layout_gb300._torch_ops cannot be loaded (%s); run "
                          "sequence_re_layout_gb300.build.build_library()" % e) from e
    _ops = _torch_ops
    return _ops


class Quantized:
    """An 8-bit matrix: ``data`` [rows, cols] float8_e4m3fn, ``scales``
    [ceil(rows / block_rows), ceil(cols / 128)] float8_e8m0fnu, where element
    (r, c) stands for ``data[r, c] * scales[r // block_rows, c // 128]``.

    Rows of ``data`` start at multiples of 16 bytes and rows of ``scales`` at
    multiples of 4; :meth:`empty` lays them out.  The call that uses a matrix
    checks it."""

    __slots__ = ("data", "scales", "block_rows")

    def __init__(self, data, scales, block_rows=1):
        self.data, self.scales, self.block_rows = data, scales, block_rows

    @classmethod
    def empty(cls, rows, cols, block_rows=1, device="cuda"):
        """Uninitialised, with rows of ``data`` padded to 16 bytes (longer ones
        than 128 to that, the cache line a product reads) and rows of ``scales``
        to 4."""
        if block_rows not in (1, BLOCK):
            raise ValueError("Quantized: block_rows must be 1 or %d" % BLOCK)
        blocks, step = -(-cols // BLOCK), 128 if cols > 128 else 16
        return cls(torch.empty_strided((rows, cols), (-(-cols // step) * step, 1), dtype=torch.float8_e4m3fn,
                                       device=device),
                   torch.empty_strided((-(-rows // block_rows), blocks), (-(-blocks // 4) * 4, 1),
                                       dtype=torch.float8_e8m0fnu, device=device), block_rows)

    @property
    def shape(self):
        return self.data.shape

    @property
    def device(self):
        return self.data.device

    def dequantize(self):
        """The values it stands for, float32 (for inspection, in plain torch)."""
        s = self.scales.float().repeat_interleave(BLOCK, 1)[:, :self.shape[1]]
        if self.block_rows > 1:
            s = s.repeat_interleave(self.block_rows, 0)[:self.shape[0]]
        return self.data.float() * s


def rmsnorm(x, weight, residual=None, eps=1e-6, quantized=True, h=None):
    """Residual addition and root-mean-square norm over the last dimension:
    ``h = x + residual``, ``y = h / sqrt(mean(h^2) + eps) * weight``.

    Returns ``(y, h, rstd)``: y as a :class:`Quantized` of [rows, cols], or with
    ``quantized=False`` as a tensor like x; h like x (x itself without a
    residual); rstd float32 [rows], which the backward takes.  ``h`` may be
    given: a buffer to write to, also that of x or of the residual.  ``weight``
    has x's element type or float32.  The residual and a given ``h`` have x's rows,
    in order, under any leading dimensions."""
    y, scales, new_h, rstd = (_ops or _load()).rmsnorm(x, weight, residual, eps, bool(quantized), h)
    return Quantized(y, scales) if quantized else y, x if new_h is None else new_h, rstd


def rmsnorm_backward(dy, h, rstd, weight, dh=None, need_dweight=True):
    """``(dx, dweight)`` of :func:`rmsnorm`: dx is the gradient of x and of the
    residual alike, with ``dh`` (the gradient that reaches h past the norm)
    added; dweight is float32, or None if not needed."""
    return (_ops or _load()).rmsnorm_backward(dy, h, rstd, weight, dh, bool(need_dweight))


def quantize(x, block_rows=1, rows=True, transposed=False):
    """x [..., cols] to 8 bits with a scale for each ``block_rows`` x 128
    values.  ``transposed`` adds the transpose [cols, rows] with scales along
    its own rows: ``(q, qt)``; with ``rows=False`` the transpose alone."""
    data, scales, data_t, scales_t = (_ops or _load()).quantize(x, block_rows, bool(rows), bool(transposed))
    q = Quantized(data, scales, block_rows) if rows else None
    if not transposed:
        return q
    qt = Quantized(data_t, scales_t, block_rows)
    return (q, qt) if rows else qt


def matmul(a, b, bias=None, out=None, out_dtype=torch.bfloat16, accumulate=False):
    """``a @ b.T`` (+ bias) of two :class:`Quantized`, [a.rows, b.rows] of
    ``out_dtype`` or into ``out``; ``accumulate`` adds to what ``out`` holds.
    The bias has the output's element type."""
    return (_ops or _load()).matmul(a.data, a.scales, a.block_rows, b.data, b.scales, b.block_rows, bias, out,
                                    out_dtype, bool(accumulate))
