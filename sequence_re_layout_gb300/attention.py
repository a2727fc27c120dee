"""Attention between the two re-layouts on torch tensors, over the C ABI of
``include/basp_attention.h``: causal, with a sliding window and a few first tokens
that stay visible (sinks).

    o, lse = attention.forward(q, k, v, window=4096, sinks=4)
    dq, dk, dv = attention.backward(do, q, k, v, o, lse, window=4096, sinks=4)
    o = attention.decode(q, k_cache, v_cache, lengths, window=4096, sinks=4)

Tensors are [batch, tokens, heads, values of a head], bfloat16 or float16, with a
head's values next to each other (a multiple of 8 of them, at most 128) and any
other strides of whole 16 bytes: a head-sharded buffer of ``seq2head`` is viewed as
``t.view(ranks * sequences, S, -1, d)``, a sequence-first one is transposed without
a copy.  k and v may have fewer heads than q, each shared by as many neighbouring
query heads.

Query i of Sq stands at position p = i + Sk - Sq among the Sk keys and sees key j if
j <= p and (j > p - window or j < sinks); ``window=None`` is all of them.  ``scale``
is that of the products, head_dim ** -0.5 if None.  What a query does not see has
no part in its results, also where it is NaN.

These functions allocate their outputs and run on the current stream; nothing
synchronises.  They are no operations of autograd (``autograd.attention`` is).
"""
from __future__ import annotations

from . import fp8


def forward(q, k, v, window=None, sinks=0, scale=None, out=None, rest=None):
    """``(o, lse)``: o like q, or into ``out``; lse float32 [batch, heads, tokens],
    the logarithm of each row's sum of exponentials, which the backward takes.  A
    query that sees nothing (more queries than keys) has o = 0 and lse = -inf.  An
    int8 tensor ``rest`` of q's shape gets what o lost when it was rounded."""
    return (fp8._ops or fp8._load()).attention(q, k, v, window, sinks, scale, out, rest)


def backward(do, q, k, v, o, lse, window=None, sinks=0, scale=None, rest=None):
    """``(dq, dk, dv)`` of :func:`forward`, contiguous, of the inputs' type.  With the
    forward's ``rest``, dq and dk are made of an o with 8 bits more: what its rounding
    adds to their error is most where a query sees few keys."""
    return (fp8._ops or fp8._load()).attention_backward(do, q, k, v, o, lse, window, sinks, scale, rest)


def decode(q, k, v, lengths, window=None, sinks=0, scale=None, out=None):
    """o [batch, heads, d] of one new token of each sequence over a cache: q
    [batch, heads, d], k and v [batch, capacity, key heads, d].  ``lengths`` int32
    [batch] on the GPU counts each sequence's tokens, the new one included, whose
    key and value are in the cache already.  Nothing of the cache past the lengths,
    or between sinks and window, is read; a sequence of no tokens has o = 0."""
    return (fp8._ops or fp8._load()).attention_decode(q, k, v, lengths, window, sinks, scale, out)
