"""8-bit norm and projections on torch tensors, over the C ABI of
``include/basp_fp8.h``: what stands before ``seq2head`` (norm and packed QKV
projection) and after ``head2seq`` (output projection).

    x8, h, rstd = fp8.rmsnorm(x, norm_weight, residual=residual)
    w8 = fp8.quantize(weight, block_rows=128)           # once, or once a step
    qkv = fp8.matmul(x8, w8, bias=bias)                 # -> seq2head_qkv

These functions allocate their outputs and run on the current stream; nothing
synchronises.  ``autograd`` has the differentiable forms.
"""
from __future__ import annotations

import torch

from . import binding

BLOCK = binding.BASP_FP8_BLOCK


def _ceil(a, b):
    return -(-a // b)


class Quantized:
    """An 8-bit matrix: ``data`` [rows, cols] float8_e4m3fn, ``scales``
    [ceil(rows / block_rows), ceil(cols / 128)] float8_e8m0fnu, where element
    (r, c) stands for ``data[r, c] * scales[r // block_rows, c // 128]``.

    Rows of ``data`` start at multiples of 16 bytes and rows of ``scales`` at
    multiples of 4, as :meth:`empty` lays them out; a matrix that came from
    elsewhere is checked by the call that uses it."""

    __slots__ = ("data", "scales", "block_rows", "_c")

    def __init__(self, data, scales, block_rows=1):
        if data.dim() != 2 or scales.dim() != 2:
            raise ValueError("Quantized: data and scales must have two dimensions")
        rows, cols = data.shape
        if block_rows not in (1, BLOCK):
            raise ValueError("Quantized: block_rows must be 1 or %d" % BLOCK)
        if data.dtype != torch.float8_e4m3fn or scales.dtype != torch.float8_e8m0fnu:
            raise ValueError("Quantized: data must be float8_e4m3fn and scales float8_e8m0fnu, got %s and %s"
                             % (data.dtype, scales.dtype))
        srows, scols = scales.shape
        if (srows, scols) != (rows if block_rows == 1 else _ceil(rows, BLOCK), _ceil(cols, BLOCK)):
            raise ValueError("Quantized: scales of shape %s do not fit data of shape %s with block_rows %d"
                             % ((srows, scols), (rows, cols), block_rows))
        if data.device != scales.device or not data.is_cuda:
            raise ValueError("Quantized: data and scales must be on one CUDA device")
        ds, ss = data.stride(), scales.stride()
        if (ds[1] != 1 and cols > 1) or (ss[1] != 1 and scols > 1):
            raise ValueError("Quantized: columns must be next to each other")
        self.data, self.scales, self.block_rows = data, scales, block_rows
        # the stride of a single row is free: any that the rules allow will do
        self._c = binding.basp_fp8_matrix(
            data.data_ptr() or None, scales.data_ptr() or None, rows, cols,
            ds[0] if rows > 1 else _ceil(cols, 16) * 16,
            ss[0] if srows > 1 else _ceil(scols, 4) * 4, block_rows)

    @classmethod
    def empty(cls, rows, cols, block_rows=1, device="cuda"):
        pitch, blocks = _ceil(cols, 16) * 16, _ceil(cols, BLOCK)
        scale_pitch = _ceil(blocks, 4) * 4
        data = torch.empty((rows, pitch), dtype=torch.float8_e4m3fn, device=device)
        scales = torch.empty((_ceil(rows, block_rows), scale_pitch), dtype=torch.float8_e8m0fnu, device=device)
        return cls(data if pitch == cols else data[:, :cols],
                   scales if scale_pitch == blocks else scales[:, :blocks], block_rows)

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


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _on_current(q, where, name):
    if q.device.index != torch.cuda.current_device():
        raise ValueError("%s: %s is on %s but the current device is cuda:%d"
                         % (where, name, q.device, torch.cuda.current_device()))


def _matrix(x):
    """[..., cols] -> [rows, cols] without a copy."""
    return x if x.dim() == 2 else x.view(-1, x.shape[-1])


def rmsnorm(x, weight, residual=None, eps=1e-6, quantized=True, h=None):
    """Residual addition and root-mean-square norm over the last dimension:
    ``h = x + residual``, ``y = h / sqrt(mean(h^2) + eps) * weight``.

    Returns ``(y, h, rstd)``: y as a :class:`Quantized` of [rows, cols], or with
    ``quantized=False`` as a tensor like x; h like x (x itself without a
    residual); rstd float32 [rows], which the backward takes.  ``h`` may be
    given: a buffer to write to, also that of x or of the residual.  ``weight``
    has x's element type or float32."""
    x2 = _matrix(x)
    rows, cols = x2.shape
    r2 = None if residual is None else _matrix(residual)
    if residual is None and h is None:
        h, h2 = x, None
    else:
        h = torch.empty_like(x) if h is None else h
        h2 = _matrix(h)
    rstd = torch.empty(rows, dtype=torch.float32, device=x.device)
    if quantized:
        y = Quantized.empty(rows, cols, 1, x.device)
        binding.basp_rmsnorm(x2, r2, weight, eps, h2, None, y._c, rstd, _stream())
    else:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        binding.basp_rmsnorm(x2, r2, weight, eps, h2, _matrix(y), None, rstd, _stream())
    return y, h, rstd


def rmsnorm_backward(dy, h, rstd, weight, dh=None, need_dweight=True):
    """``(dx, dweight)`` of :func:`rmsnorm`: dx is the gradient of x and of the
    residual alike, with ``dh`` (the gradient that reaches h past the norm)
    added; dweight is float32, or None if not needed."""
    dy2 = _matrix(dy)
    rows, cols = dy2.shape
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    dweight = workspace = None
    if need_dweight:
        dweight = torch.empty(cols, dtype=torch.float32, device=dy.device)
        workspace = torch.empty(binding.basp_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8,
                                device=dy.device)
    binding.basp_rmsnorm_backward(dy2, _matrix(h), rstd, weight, None if dh is None else _matrix(dh),
                                  _matrix(dx), dweight, workspace, _stream())
    return dx, dweight


def quantize(x, block_rows=1, rows=True, transposed=False):
    """x [..., cols] to 8 bits with a scale for each ``block_rows`` x 128
    values.  ``transposed`` adds the transpose [cols, rows] with scales along
    its own rows: ``(q, qt)``; with ``rows=False`` the transpose alone."""
    x2 = _matrix(x)
    q = Quantized.empty(*x2.shape, block_rows, x.device) if rows else None
    qt = Quantized.empty(x2.shape[1], x2.shape[0], block_rows, x.device) if transposed else None
    binding.basp_quantize_fp8(x2, q._c if rows else None, qt._c if transposed else None, _stream())
    return (q, qt) if rows and transposed else q if rows else qt


def matmul(a, b, bias=None, out=None, out_dtype=torch.bfloat16, accumulate=False):
    """``a @ b.T`` (+ bias) of two :class:`Quantized`, [a.rows, b.rows] of
    ``out_dtype`` or into ``out``; ``accumulate`` adds to what ``out`` holds.
    The bias has the output's element type."""
    if accumulate and out is None:
        raise ValueError("matmul: accumulate needs out")
    _on_current(a, "matmul", "a")
    if b.device != a.device:
        raise ValueError("matmul: a is on %s and b on %s" % (a.device, b.device))
    if a.shape[1] != b.shape[1]:
        raise ValueError("matmul: a has %d columns and b %d" % (a.shape[1], b.shape[1]))
    if out is None:
        out = torch.empty((a.shape[0], b.shape[0]), dtype=out_dtype, device=a.device)
    binding.basp_matmul_fp8(a._c, b._c, bias, out, accumulate, _stream())
    return out
