"""PyTorch autograd wrappers over the C ABI, for training loops.

The re-layout is a permutation, so its gradient is the inverse permutation:
the backward of seq2head is head2seq of the gradients, and the backward of
head2seq is seq2head.  Both directions run in the library's kernels; this
module only allocates the outputs with torch and routes the gradients.

    L = basp.Layout(B, S, Hq, Hkv, d, N, K, "bf16")
    q_h, k_h, v_h = seq2head(L, q, k, v)     # before attention
    o_s = head2seq(L, o_h)                   # after attention
    q_h, k_h, v_h = seq2head_qkv(L, qkv)     # from a fused QKV projection

Inputs are virtual-rank buffers (flat, or any contiguous shape with the right
number of elements); outputs are flat tensors of the same dtype and device.

The projections on both sides of the re-layout, in 8 bits (``fp8`` has the
operators they are made of):

    y, h = rmsnorm(x, norm_weight, residual=r)                      # 16 bits out
    qkv, h = rmsnorm_linear_fp8(x, norm_weight, wqkv, bqkv, residual=r)
    out = linear_fp8(o, wo)

Their gradients treat the rounding to 8 bits as the identity, and round the
operands of the gradients' products the same way: with dY in 8 bits along its
rows, dX = dY W; with dY and X in 8 bits along the tokens, dW = dY^T X.

As for any torch code, a CUDA graph that captures a backward pass captures its
forward pass too, with no other graph of the same parameters alive.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding, fp8


def _stream():
    return torch.cuda.current_stream()


def _contig(t):
    return None if t is None else t.contiguous()


class _Seq2Head(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layout, q, k, v):
        ctx.layout = layout
        ins = [_contig(t) for t in (q, k, v)]
        outs = [None if t is None else torch.empty_like(t).view(-1) for t in ins]
        binding.basp_seq2head(layout.handle, "fused", *ins, *outs, stream=_stream())
        return tuple(outs)

    @staticmethod
    def backward(ctx, dq, dk, dv):
        grads = [_contig(g) for g in (dq, dk, dv)]
        outs = [None if g is None else torch.empty_like(g) for g in grads]
        if any(g is not None for g in grads):
            binding.basp_head2seq(ctx.layout.handle, "fused", *grads, *outs,
                                  stream=_stream())
        return (None, *outs)


class _Head2Seq(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layout, o):
        ctx.layout = layout
        o = o.contiguous()
        out = torch.empty_like(o).view(-1)
        binding.basp_head2seq(layout.handle, "fused", o, None, None, out, None, None,
                              stream=_stream())
        return out

    @staticmethod
    def backward(ctx, do):
        do = do.contiguous()
        out = torch.empty_like(do)
        binding.basp_seq2head(ctx.layout.handle, "fused", do, None, None, out, None,
                              None, stream=_stream())
        return None, out


def seq2head(layout, q, k=None, v=None):
    """seq-sharded Q (Hq heads) and optional K, V (Hkv heads) -> head-sharded,
    differentiable.  Returns a tuple (q_h, k_h, v_h) with None where an input
    was None."""
    return _Seq2Head.apply(layout, q, k, v)


def head2seq(layout, o):
    """head-sharded attention output O (Hq heads) -> seq-sharded,
    differentiable."""
    return _Head2Seq.apply(layout, o)


class _Seq2HeadQKV(torch.autograd.Function):
    @staticmethod
    def forward(ctx, layout, qkv):
        ctx.layout = layout
        qkv = qkv.contiguous()
        ctx.packed_shape = qkv.shape
        esz = qkv.element_size()
        i = layout.info
        outs = [torch.empty(n // esz, dtype=qkv.dtype, device=qkv.device)
                for n in (i["bytes_q"], i["bytes_kv"], i["bytes_kv"])]
        binding.basp_seq2head_qkv(layout.handle, qkv, *outs, stream=_stream())
        return tuple(outs)

    @staticmethod
    def backward(ctx, dq, dk, dv):
        i = ctx.layout.info
        ref = next(g for g in (dq, dk, dv) if g is not None)
        esz = ref.element_size()
        # the packed gradient has every head range: a missing one is zero
        grads = [torch.zeros(n // esz, dtype=ref.dtype, device=ref.device) if g is None
                 else g.contiguous()
                 for g, n in zip((dq, dk, dv), (i["bytes_q"], i["bytes_kv"], i["bytes_kv"]))]
        out = torch.empty(ctx.packed_shape, dtype=ref.dtype, device=ref.device)
        binding.basp_head2seq_qkv(ctx.layout.handle, *grads, out, stream=_stream())
        return None, out


def seq2head_qkv(layout, qkv):
    """seq-sharded packed QKV (each token row holds the Hq query heads, then
    the Hkv key heads, then the Hkv value heads: a fused QKV projection's
    output) -> head-sharded Q, K, V, differentiable.  The backward packs the
    three gradients into one seq-sharded gradient of the packed input."""
    return _Seq2HeadQKV.apply(layout, qkv)


# ---- 8-bit projections -------------------------------------------------------
#
# Without gradient mode the functions below keep nothing and quantise no
# transposes; a weight may then be a fp8.Quantized, rounded once for many calls.

def _rows(t):
    """[..., cols] -> [rows, cols]."""
    return t.flatten(0, -2) if t.dim() > 1 else t.unsqueeze(0)


def _shaped(grad, shape):
    """The gradient of the residual, which may have x's rows under other leading
    dimensions."""
    return grad if grad is None or grad.shape == shape else grad.reshape(shape)


def _saved(q):
    return (None, None) if q is None else (q.data, q.scales)


def _quantized_weight(weight, transposed):
    """(weight, its transpose or None) in 8 bits.  128 x 128 blocks: both
    directions hold the same values, so dX = dY W sees the W of the forward."""
    if transposed:
        return fp8.quantize(weight, block_rows=fp8.BLOCK, transposed=True)
    return fp8.quantize(weight, block_rows=fp8.BLOCK), None


def _product_grads(dy, weight_t, x_t, weight_dtype, need_bias):
    """(dx, dweight, dbias) of y = x weight^T + bias; dx without weight_t and
    dweight without x_t are None."""
    d = d_t = None
    if weight_t is not None and x_t is not None:
        d, d_t = fp8.quantize(dy, transposed=True)
    elif weight_t is not None:
        d = fp8.quantize(dy)
    elif x_t is not None:
        d_t = fp8.quantize(dy, rows=False, transposed=True)
    return (None if d is None else fp8.matmul(d, weight_t, out_dtype=dy.dtype),
            None if d_t is None else fp8.matmul(d_t, x_t, out_dtype=weight_dtype),
            dy.sum(0, dtype=torch.float32).to(dy.dtype) if need_bias else None)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, rstd = fp8.rmsnorm(x, weight, residual, eps, quantized=False)
        ctx.save_for_backward(h, rstd, weight)
        ctx.residual_shape = None if residual is None else residual.shape
        ctx.set_materialize_grads(False)
        return y, h.view_as(h) if residual is None else h       # an input comes back as a view of it

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, rstd, weight = ctx.saved_tensors
        need_x, need_w, need_residual, _ = ctx.needs_input_grad
        dx, dw = dh, None
        if dy is not None:
            dx, dw = fp8.rmsnorm_backward(dy.contiguous(), h, rstd, weight, _contig(dh), need_w)
        return (dx if need_x else None, None if dw is None else dw.to(weight.dtype),
                _shaped(dx, ctx.residual_shape) if need_residual else None, None)


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """``(y, h)`` with h = x + residual and y = h / sqrt(mean(h^2) + eps) *
    weight over the last dimension, differentiable.  h carries the residual
    stream on: its gradient joins the norm's in one kernel.  y and h have x's shape;
    the residual has x's rows, in order, under any leading dimensions."""
    return _RmsNorm.apply(x, weight, residual, eps)


class _LinearFp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        need_x, need_w, _ = ctx.needs_input_grad
        w, w_t = _quantized_weight(weight, need_x)
        q, q_t = fp8.quantize(_rows(x), transposed=True) if need_w else (fp8.quantize(_rows(x)), None)
        ctx.save_for_backward(*_saved(w_t), *_saved(q_t))
        ctx.x_shape, ctx.weight_dtype = x.shape, weight.dtype
        return fp8.matmul(q, w, bias=bias, out_dtype=x.dtype).view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        wd, ws, xd, xs = ctx.saved_tensors
        dx, dw, db = _product_grads(_rows(dy).contiguous(),
                                    None if wd is None else fp8.Quantized(wd, ws, fp8.BLOCK),
                                    None if xd is None else fp8.Quantized(xd, xs),
                                    ctx.weight_dtype, ctx.needs_input_grad[2])
        return None if dx is None else dx.view(ctx.x_shape), dw, db


def linear_fp8(x, weight, bias=None):
    """``x @ weight.T (+ bias)`` with x [..., in] and weight [out, in] rounded to
    8 bits, differentiable.  The result, the bias and the gradient of x have x's
    element type, the gradient of the weight has the weight's (a 32-bit master
    weight gets a 32-bit gradient)."""
    if not torch.is_grad_enabled():
        q = fp8.quantize(_rows(x))
        w = weight if isinstance(weight, fp8.Quantized) else _quantized_weight(weight, False)[0]
        return fp8.matmul(q, w, bias=bias, out_dtype=x.dtype).view(*x.shape[:-1], w.shape[0])
    _refuse_quantized(weight)
    return _LinearFp8.apply(x, weight, bias)


class _RmsNormLinearFp8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_weight, weight, bias, residual, eps):
        need = ctx.needs_input_grad
        w, w_t = _quantized_weight(weight, need[0] or need[1] or need[4])
        q, h, rstd = fp8.rmsnorm(x, norm_weight, residual, eps)
        ctx.save_for_backward(h, rstd, norm_weight, *_saved(w_t))
        ctx.eps, ctx.weight_dtype = eps, weight.dtype
        ctx.residual_shape = None if residual is None else residual.shape
        ctx.set_materialize_grads(False)
        y = fp8.matmul(q, w, bias=bias, out_dtype=x.dtype).view(*x.shape[:-1], weight.shape[0])
        return y, h.view_as(h) if residual is None else h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, rstd, norm_weight, wd, ws = ctx.saved_tensors
        need_x, need_nw, need_w, need_b, need_residual, _ = ctx.needs_input_grad
        dx, dnw, dw, db = dh, None, None, None
        if dy is not None:
            x_t = None
            if need_w:
                # the 8-bit rows of the forward have their scales along the wrong
                # side for this sum over the tokens: the norm again, from h (rounded
                # to 16 bits on the way, 2^-8 beside the 2^-4 of the 8 bits)
                y, _, _ = fp8.rmsnorm(h, norm_weight, None, ctx.eps, quantized=False)
                x_t = fp8.quantize(_rows(y), rows=False, transposed=True)
            dn, dw, db = _product_grads(_rows(dy).contiguous(),
                                        None if wd is None else fp8.Quantized(wd, ws, fp8.BLOCK), x_t,
                                        ctx.weight_dtype, need_b)
            if dn is not None:
                dx, dnw = fp8.rmsnorm_backward(dn.view(h.shape), h, rstd, norm_weight, _contig(dh), need_nw)
        return (dx if need_x else None, None if dnw is None else dnw.to(norm_weight.dtype), dw, db,
                _shaped(dx, ctx.residual_shape) if need_residual else None, None)


def rmsnorm_linear_fp8(x, norm_weight, weight, bias=None, residual=None, eps=1e-6):
    """``(y, h)``: :func:`rmsnorm` and :func:`linear_fp8` of its result, whose
    values pass from one to the other in 8 bits.  The backward keeps h, one
    number a row and the 8-bit transpose of the weight."""
    if not torch.is_grad_enabled():
        q, h, _ = fp8.rmsnorm(x, norm_weight, residual, eps)
        w = weight if isinstance(weight, fp8.Quantized) else _quantized_weight(weight, False)[0]
        return fp8.matmul(q, w, bias=bias, out_dtype=x.dtype).view(*x.shape[:-1], w.shape[0]), h
    _refuse_quantized(weight)
    return _RmsNormLinearFp8.apply(x, norm_weight, weight, bias, residual, eps)


def _refuse_quantized(weight):
    if isinstance(weight, fp8.Quantized):
        raise TypeError("an 8-bit weight has no gradient: call under torch.no_grad(), or pass the 16/32-bit weight")
