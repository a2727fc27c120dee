"""ctypes binding of ``libbasp.so`` (declared in ``include/basp.h``,
``include/basp_fp8.h``, ``include/basp_attention.h`` and ``include/basp_optim.h``).

Argument marshalling only: every function here takes Python ints or torch
tensors, turns them into the C-ABI's pointers and sizes, calls the library and
raises :class:`BaspError` on a non-OK status.  The re-layout itself runs in the
library's CUDA kernels; there is no other implementation behind these names.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
# BASP_LIBRARY=debug selects the bounds-checking build (libbasp_debug.so);
# BASP_LIBRARY_PATH names any other build of the same sources explicitly
LIB_PATH = os.environ.get("BASP_LIBRARY_PATH") or os.path.join(
    PKG, "libbasp_debug.so" if os.environ.get("BASP_LIBRARY") == "debug" else "libbasp.so")

# enums of basp.h
BASP_DTYPE_BF16, BASP_DTYPE_FP32, BASP_DTYPE_FP16, BASP_DTYPE_FP8 = 0, 1, 2, 3
BASP_ALGO_FUSED, BASP_ALGO_THREE_PASS, BASP_ALGO_THREE_PASS_ELIDE = 0, 1, 2
BASP_ORDER_BSHD, BASP_ORDER_SBHD = 0, 1
(BASP_OK, BASP_ERR_INVALID_ARG, BASP_ERR_DIVISIBILITY, BASP_ERR_BATCH_GT_RANKS,
 BASP_ERR_ALIGNMENT, BASP_ERR_ALIASING, BASP_ERR_WORKSPACE, BASP_ERR_CUDA,
 BASP_ERR_TOO_LARGE) = range(9)

DTYPE_CODES = {"bf16": BASP_DTYPE_BF16, "fp32": BASP_DTYPE_FP32,
               "fp16": BASP_DTYPE_FP16, "fp8": BASP_DTYPE_FP8}
ALGO_CODES = {"fused": BASP_ALGO_FUSED, "three_pass": BASP_ALGO_THREE_PASS,
              "three_pass_elide": BASP_ALGO_THREE_PASS_ELIDE}
ORDER_CODES = {"bshd": BASP_ORDER_BSHD, "sbhd": BASP_ORDER_SBHD}

# every symbol include/basp.h declares
EXPORTS = ("basp_layout_create", "basp_layout_create_ex", "basp_layout_query",
           "basp_layout_destroy", "basp_seq2head", "basp_head2seq",
           "basp_seq2head_qkv", "basp_head2seq_qkv", "basp_seq2head_host",
           "basp_head2seq_host", "basp_seq2head_noalloc", "basp_status_string")

# every symbol include/basp_fp8.h declares
FP8_EXPORTS = ("basp_rmsnorm", "basp_rmsnorm_backward", "basp_rmsnorm_backward_workspace",
               "basp_quantize_fp8", "basp_matmul_fp8", "basp_matmul_fp8_timeouts",
               "basp_layernorm", "basp_layernorm_backward", "basp_layernorm_backward_workspace")

# every symbol include/basp_attention.h declares
ATTENTION_EXPORTS = ("basp_attention", "basp_attention_backward", "basp_attention_backward_workspace",
                     "basp_attention_decode", "basp_attention_decode_workspace", "basp_attention_timeouts")

# every symbol include/basp_optim.h declares
OPTIM_EXPORTS = ("basp_adamw", "basp_adamw_each")

# values that share a scale along a row of an 8-bit matrix
BASP_FP8_BLOCK = 128

# size of the library's built-in scratch for basp_seq2head_noalloc
BASP_NOALLOC_SCRATCH_BYTES = 32 << 20


class basp_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "B", "S", "Hq", "Hkv", "d", "N", "K", "groups", "seqs_per_group",
        "tokens_per_rank", "elem_size", "elems_per_rank_q", "elems_per_rank_kv",
        "peers", "bytes_per_peer_q", "bytes_per_peer_kv", "bytes_q", "bytes_kv",
        "workspace_bytes", "staging_bytes", "foil_tokens_per_rank", "order",
        "bytes_qkv_packed")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class basp_layout_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "S", "Hq", "Hkv", "d", "N", "K")] + \
        [("dtype", ctypes.c_int), ("order", ctypes.c_int)]


class basp_fp8_matrix(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p)] + \
        [(n, ctypes.c_int64) for n in ("rows", "cols", "pitch", "scale_pitch", "block_rows")]


class basp_attention_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("batch", "q_len", "k_len", "q_heads", "k_heads", "head_dim", "window",
                                              "sinks")] + [("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class basp_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + \
        [(n, ctypes.c_int64) for n in ("stride_batch", "stride_seq", "stride_head")]


class basp_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "m_scales", "v_scales")] + \
        [("n", ctypes.c_int64), ("dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int)]


class basp_adamw_options(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
        [("step", ctypes.c_int64), ("step_at", ctypes.c_void_p), ("seed", ctypes.c_uint32)]


class BaspError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, basp_status_string(status), status))


_lib = None


def load_library():
    """Load the in-tree ``libbasp.so``.  There is no fallback: a missing
    library is an error."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libbasp.so is not built (expected at %s); run "
            "sequence_re_layout_gb300.build.build_library()" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.basp_layout_create.argtypes = [i64] * 7 + [ctypes.c_int, ctypes.POINTER(vp)]
    lib.basp_layout_create.restype = ctypes.c_int
    lib.basp_layout_create_ex.argtypes = [ctypes.POINTER(basp_layout_desc),
                                          ctypes.POINTER(vp)]
    lib.basp_layout_create_ex.restype = ctypes.c_int
    lib.basp_layout_query.argtypes = [vp, ctypes.POINTER(basp_info)]
    lib.basp_layout_query.restype = ctypes.c_int
    lib.basp_layout_destroy.argtypes = [vp]
    lib.basp_layout_destroy.restype = None
    for name in ("basp_seq2head", "basp_head2seq"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, ctypes.c_int] + [vp] * 6 + [vp, sz, vp]
        fn.restype = ctypes.c_int
    for name in ("basp_seq2head_host", "basp_head2seq_host"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, ctypes.c_int] + [vp] * 6 + [vp, sz, vp, sz, vp]
        fn.restype = ctypes.c_int
    lib.basp_seq2head_qkv.argtypes = [vp] * 6
    lib.basp_seq2head_qkv.restype = ctypes.c_int
    lib.basp_head2seq_qkv.argtypes = [vp] * 6
    lib.basp_head2seq_qkv.restype = ctypes.c_int
    lib.basp_seq2head_noalloc.argtypes = [vp] + [vp] * 6 + [vp]
    lib.basp_seq2head_noalloc.restype = ctypes.c_int
    ci, mp = ctypes.c_int, ctypes.POINTER(basp_fp8_matrix)
    lib.basp_rmsnorm.argtypes = [ci, i64, i64, vp, i64, vp, i64, vp, ci, ctypes.c_float,
                                 vp, i64, vp, i64, mp, vp, vp]
    lib.basp_rmsnorm.restype = ci
    lib.basp_rmsnorm_backward.argtypes = [ci, i64, i64, vp, i64, vp, i64, vp, vp, ci, vp, i64,
                                          vp, i64, vp, vp, sz, vp]
    lib.basp_rmsnorm_backward.restype = ci
    lib.basp_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.basp_rmsnorm_backward_workspace.restype = i64
    lib.basp_quantize_fp8.argtypes = [ci, i64, i64, vp, i64, mp, mp, vp]
    lib.basp_quantize_fp8.restype = ci
    lib.basp_matmul_fp8.argtypes = [mp, mp, vp, ci, ci, vp, i64, vp]
    lib.basp_matmul_fp8.restype = ci
    lib.basp_matmul_fp8_timeouts.argtypes = [ctypes.POINTER(ctypes.c_ulonglong)]
    lib.basp_matmul_fp8_timeouts.restype = ci
    lib.basp_layernorm.argtypes = [ci, i64, i64, vp, i64, vp, i64, vp, vp, ci, ctypes.c_float,
                                   vp, i64, vp, i64, mp, vp, vp, vp]
    lib.basp_layernorm.restype = ci
    lib.basp_layernorm_backward.argtypes = [ci, i64, i64, vp, i64, vp, i64, vp, vp, vp, ci, vp, i64,
                                            vp, i64, vp, vp, vp, sz, vp]
    lib.basp_layernorm_backward.restype = ci
    lib.basp_layernorm_backward_workspace.argtypes = [i64, i64]
    lib.basp_layernorm_backward_workspace.restype = i64
    dp, hp = ctypes.POINTER(basp_attention_desc), ctypes.POINTER(basp_heads)
    lib.basp_attention.argtypes = [dp] + [hp] * 5 + [vp, vp]
    lib.basp_attention.restype = ci
    lib.basp_attention_backward.argtypes = [dp] + [hp] * 5 + [vp] + [hp] * 4 + [vp, sz, vp]
    lib.basp_attention_backward.restype = ci
    lib.basp_attention_decode.argtypes = [dp] + [hp] * 3 + [vp, hp, vp, sz, vp]
    lib.basp_attention_decode.restype = ci
    for name in ("basp_attention_backward_workspace", "basp_attention_decode_workspace"):
        getattr(lib, name).argtypes = [dp]
        getattr(lib, name).restype = i64
    lib.basp_attention_timeouts.argtypes = [ctypes.POINTER(ctypes.c_ulonglong)]
    lib.basp_attention_timeouts.restype = ci
    lib.basp_adamw.argtypes = [ctypes.POINTER(basp_adamw_tensor), i64, ctypes.POINTER(basp_adamw_options), vp]
    lib.basp_adamw.restype = ci
    lib.basp_adamw_each.argtypes = [ctypes.POINTER(basp_adamw_tensor), ctypes.POINTER(vp),
                                    ctypes.POINTER(ctypes.c_uint32), i64, ctypes.POINTER(basp_adamw_options), vp]
    lib.basp_adamw_each.restype = ci
    if hasattr(lib, "basp_debug_bounds_violations"):
        lib.basp_debug_bounds_violations.argtypes = [ctypes.POINTER(ctypes.c_ulonglong)]
        lib.basp_debug_bounds_violations.restype = ctypes.c_int
    lib.basp_status_string.argtypes = [ctypes.c_int]
    lib.basp_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(x):
    """A device/host address from None, an int or a tensor."""
    if x is None:
        return None
    if isinstance(x, int):
        return x or None
    return x.data_ptr() or None


# layout handle -> basp_info dict, so tensor arguments can be checked cheaply
_INFO = {}


def _info(layout):
    i = _INFO.get(layout)
    if i is None and layout:
        i = basp_layout_query(layout)
    return i


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _tptr(x, need, where, name, place, cur=None):
    """Address of a buffer argument.  Raw ints pass through unchecked; a tensor
    must be contiguous, hold at least `need` bytes, and live where the call
    reads it: "device" (a CUDA tensor on the current device, or page-locked
    host memory, which the kernels reach over the host link) or "host" (CPU
    memory)."""
    if x is None or isinstance(x, int):
        return _ptr(x)
    if not x.is_contiguous():
        raise ValueError("%s: %s must be contiguous" % (where, name))
    if need is not None and x.nbytes < need:
        raise ValueError("%s: %s holds %d bytes, the layout needs %d"
                         % (where, name, x.nbytes, need))
    if place == "device":
        if x.is_cuda:
            # the library launches on the current device (and takes its
            # built-in scratch there), so a tensor on another GPU would be
            # reached across devices: refuse it
            if cur is None:
                cur = _current_device()
            if x.device.index != cur:
                raise ValueError("%s: %s is on cuda:%s but the current device is "
                                 "cuda:%d; make its device current first"
                                 % (where, name, x.device.index, cur))
        elif not x.is_pinned():
            raise ValueError("%s: %s must be a CUDA tensor or page-locked host "
                             "memory" % (where, name))
    elif x.is_cuda:
        raise ValueError("%s: %s must be in host memory" % (where, name))
    return x.data_ptr() or None


def _triple(layout, where, names, bufs, place):
    """Check the (Hq, Hkv, Hkv) buffer triple of one call."""
    i = _info(layout)
    need = (i["bytes_q"], i["bytes_kv"], i["bytes_kv"]) if i else (None,) * 3
    # the current device, asked once for the whole triple
    cur = None
    if place == "device" and any(getattr(b, "is_cuda", False) for b in bufs):
        cur = _current_device()
    return [_tptr(b, n, where, nm, place, cur) for b, n, nm in zip(bufs, need, names)]


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s or None
    return s.cuda_stream or None


def _check(status, where):
    if status != BASP_OK:
        raise BaspError(status, where)


def basp_status_string(status: int) -> str:
    return load_library().basp_status_string(int(status)).decode()


def basp_layout_create(B, S, Hq, Hkv, d, N, K, dtype="bf16") -> int:
    """Create a layout handle (an opaque int).  ``K = 0`` asks for the BASP
    rule K = N/B.  ``dtype`` is "bf16", "fp16", "fp32" or the enum value."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    h = ctypes.c_void_p()
    _check(load_library().basp_layout_create(B, S, Hq, Hkv, d, N, K, code,
                                             ctypes.byref(h)),
           "basp_layout_create")
    _INFO[h.value] = basp_layout_query(h.value)
    return h.value


def basp_layout_create_ex(B, S, Hq, Hkv, d, N, K, dtype="bf16", order="bshd") -> int:
    """Create a layout handle with a token order ("bshd" batch-first or
    "sbhd" sequence-first, or the enum value)."""
    desc = basp_layout_desc(
        B, S, Hq, Hkv, d, N, K,
        DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype),
        ORDER_CODES[order] if isinstance(order, str) else int(order))
    h = ctypes.c_void_p()
    _check(load_library().basp_layout_create_ex(ctypes.byref(desc), ctypes.byref(h)),
           "basp_layout_create_ex")
    _INFO[h.value] = basp_layout_query(h.value)
    return h.value


def basp_layout_query(layout: int) -> dict:
    info = basp_info()
    _check(load_library().basp_layout_query(layout, ctypes.byref(info)),
           "basp_layout_query")
    return info.as_dict()


def basp_layout_destroy(layout: int) -> None:
    _INFO.pop(layout, None)
    load_library().basp_layout_destroy(layout)


def _algo(a):
    return ALGO_CODES[a] if isinstance(a, str) else int(a)


def _nbytes(x):
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.numel() * x.element_size()


def basp_seq2head(layout, algo, q, k, v, q_out, k_out, v_out,
                  workspace=None, workspace_bytes=None, stream=None):
    """seq-sharded -> head-sharded (device buffers); see ``basp.h``."""
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    w = "basp_seq2head"
    a = _triple(layout, w, ("q", "k", "v"), (q, k, v), "device")
    b = _triple(layout, w, ("q_out", "k_out", "v_out"), (q_out, k_out, v_out), "device")
    _check(load_library().basp_seq2head(
        layout, _algo(algo), *a, *b,
        _tptr(workspace, None, w, "workspace", "device"), wb, _stream(stream)), w)


def basp_head2seq(layout, algo, o, k, v, o_out, k_out, v_out,
                  workspace=None, workspace_bytes=None, stream=None):
    """head-sharded -> seq-sharded (device buffers); see ``basp.h``."""
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    w = "basp_head2seq"
    a = _triple(layout, w, ("o", "k", "v"), (o, k, v), "device")
    b = _triple(layout, w, ("o_out", "k_out", "v_out"), (o_out, k_out, v_out), "device")
    _check(load_library().basp_head2seq(
        layout, _algo(algo), *a, *b,
        _tptr(workspace, None, w, "workspace", "device"), wb, _stream(stream)), w)


def basp_seq2head_host(layout, algo, q, k, v, q_out, k_out, v_out, staging,
                       staging_bytes=None, workspace=None,
                       workspace_bytes=None, stream=None):
    """Host buffers in and out, device ``staging``; see ``basp.h``."""
    sb = _nbytes(staging) if staging_bytes is None else staging_bytes
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    w = "basp_seq2head_host"
    a = _triple(layout, w, ("q", "k", "v"), (q, k, v), "host")
    b = _triple(layout, w, ("q_out", "k_out", "v_out"), (q_out, k_out, v_out), "host")
    _check(load_library().basp_seq2head_host(
        layout, _algo(algo), *a, *b, _tptr(staging, None, w, "staging", "device"), sb,
        _tptr(workspace, None, w, "workspace", "device"), wb, _stream(stream)), w)


def basp_head2seq_host(layout, algo, o, k, v, o_out, k_out, v_out, staging,
                       staging_bytes=None, workspace=None,
                       workspace_bytes=None, stream=None):
    """Host buffers in and out, device ``staging``; see ``basp.h``."""
    sb = _nbytes(staging) if staging_bytes is None else staging_bytes
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    w = "basp_head2seq_host"
    a = _triple(layout, w, ("o", "k", "v"), (o, k, v), "host")
    b = _triple(layout, w, ("o_out", "k_out", "v_out"), (o_out, k_out, v_out), "host")
    _check(load_library().basp_head2seq_host(
        layout, _algo(algo), *a, *b, _tptr(staging, None, w, "staging", "device"), sb,
        _tptr(workspace, None, w, "workspace", "device"), wb, _stream(stream)), w)


def basp_debug_bounds_violations() -> int:
    """Debug build only: read and clear the count of out-of-bounds accesses
    the kernels skipped on the current device (synchronises it)."""
    lib = load_library()
    if not hasattr(lib, "basp_debug_bounds_violations"):
        raise RuntimeError("the loaded library is not the bounds-checking build "
                           "(set BASP_LIBRARY=debug before importing)")
    n = ctypes.c_ulonglong()
    _check(lib.basp_debug_bounds_violations(ctypes.byref(n)), "basp_debug_bounds_violations")
    return n.value


def basp_seq2head_qkv(layout, qkv, q_out, k_out, v_out, stream=None):
    """Packed seq-sharded QKV -> head-sharded Q, K, V; see ``basp.h``."""
    w = "basp_seq2head_qkv"
    i = _info(layout)
    p = _tptr(qkv, i["bytes_qkv_packed"] if i else None, w, "qkv", "device")
    b = _triple(layout, w, ("q_out", "k_out", "v_out"), (q_out, k_out, v_out), "device")
    _check(load_library().basp_seq2head_qkv(layout, p, *b, _stream(stream)), w)


def basp_head2seq_qkv(layout, q, k, v, qkv_out, stream=None):
    """Head-sharded Q, K, V -> packed seq-sharded QKV; see ``basp.h``."""
    w = "basp_head2seq_qkv"
    i = _info(layout)
    a = _triple(layout, w, ("q", "k", "v"), (q, k, v), "device")
    p = _tptr(qkv_out, i["bytes_qkv_packed"] if i else None, w, "qkv_out", "device")
    _check(load_library().basp_head2seq_qkv(layout, *a, p, _stream(stream)), w)


def basp_seq2head_noalloc(layout, q, k, v, q_out, k_out, v_out, stream=None):
    """seq-sharded -> head-sharded through the three-pass path, using the
    library's built-in scratch instead of a workspace: for callers that cannot
    allocate device memory.  See ``basp.h`` for the size limit and the rule
    that calls sharing the scratch must not overlap on the GPU."""
    w = "basp_seq2head_noalloc"
    a = _triple(layout, w, ("q", "k", "v"), (q, k, v), "device")
    b = _triple(layout, w, ("q_out", "k_out", "v_out"), (q_out, k_out, v_out), "device")
    _check(load_library().basp_seq2head_noalloc(layout, *a, *b, _stream(stream)), w)


# ---- the 8-bit projections (include/basp_fp8.h) ----------------------------

# Calls here take microseconds on the GPU, so the checks are kept to a few
# attribute reads a tensor; each refuses with ValueError before the C call.

_FP8_DTYPES = {}       # torch element type -> basp_dtype
_F32 = None            # torch.float32


def _fp8_types():
    global _F32
    import torch
    _FP8_DTYPES.update({torch.bfloat16: BASP_DTYPE_BF16, torch.float16: BASP_DTYPE_FP16,
                        torch.float32: BASP_DTYPE_FP32})
    _F32 = torch.float32


def fp8_dtype_code(dtype) -> int:
    """basp_dtype of a torch element type that the 8-bit operators take or
    give (bfloat16, float16, float32)."""
    if not _FP8_DTYPES:
        _fp8_types()
    code = _FP8_DTYPES.get(dtype)
    if code is None:
        raise ValueError("element type must be bfloat16, float16 or float32, got %s" % (dtype,))
    return code


def _wrong(x, where, name, shape, dtype, cur):
    if x.get_device() != cur:
        what = "must be on the current device cuda:%d, it is on %s" % (cur, x.device)
    elif x.dtype != dtype:
        what = "must be %s, got %s" % (dtype, x.dtype)
    elif tuple(x.shape) != shape:
        what = "must have shape %s, got %s" % (shape, tuple(x.shape))
    else:
        what = "must have its columns next to each other, got strides %s" % (tuple(x.stride()),)
    raise ValueError("%s: %s %s" % (where, name, what))


def _rows(x, where, name, shape, dtype, cur):
    """(address, row stride) of a CUDA matrix of this (rows, cols) with unit
    column stride and the given element type; (None, 0) for None."""
    if x is None:
        return None, 0
    if x.get_device() != cur or x.dtype != dtype or x.shape != shape:
        _wrong(x, where, name, shape, dtype, cur)
    s0, s1 = x.stride()
    if s1 != 1 and shape[1] > 1:
        _wrong(x, where, name, shape, dtype, cur)
    # the stride of a single row says nothing
    return x.data_ptr() or None, s0 if shape[0] > 1 else shape[1]


def _vector(x, where, name, n, dtype, cur):
    """Address of a contiguous CUDA vector of n elements, or None."""
    if x is None:
        return None
    if x.get_device() != cur or x.dtype != dtype or x.shape != (n,) or (n > 1 and x.stride() != (1,)):
        _wrong(x, where, name, (n,), dtype, cur)
    return x.data_ptr() or None


def _2d(x, where, name):
    if x.dim() != 2:
        raise ValueError("%s: %s must have two dimensions, got shape %s" % (where, name, tuple(x.shape)))
    return tuple(x.shape)


def basp_rmsnorm(x, residual, weight, eps, h=None, y=None, q=None, rstd=None, stream=None):
    """Residual addition + root-mean-square norm; see ``basp_fp8.h``.  ``q`` is
    a :class:`basp_fp8_matrix`, everything else a tensor or None."""
    w = "basp_rmsnorm"
    shape, t = _2d(x, w, "x"), x.dtype
    code, wcode, cur = fp8_dtype_code(t), fp8_dtype_code(weight.dtype), _current_device()
    xp, xs = _rows(x, w, "x", shape, t, cur)
    rp, rs = _rows(residual, w, "residual", shape, t, cur)
    hp, hs = _rows(h, w, "h", shape, t, cur)
    yp, ys = _rows(y, w, "y", shape, t, cur)
    st = load_library().basp_rmsnorm(
        code, shape[0], shape[1], xp, xs, rp, rs, _vector(weight, w, "weight", shape[1], weight.dtype, cur),
        wcode, eps, hp, hs, yp, ys, q, _vector(rstd, w, "rstd", shape[0], _F32, cur), _stream(stream))
    if st:
        _check(st, w)


def basp_rmsnorm_backward_workspace(rows: int, cols: int) -> int:
    return load_library().basp_rmsnorm_backward_workspace(rows, cols)


def basp_rmsnorm_backward(dy, h, rstd, weight, dh, dx, dweight=None, workspace=None, stream=None):
    """Gradient of :func:`basp_rmsnorm`; see ``basp_fp8.h``."""
    w = "basp_rmsnorm_backward"
    shape, t = _2d(dy, w, "dy"), dy.dtype
    code, wcode, cur = fp8_dtype_code(t), fp8_dtype_code(weight.dtype), _current_device()
    yp, ys = _rows(dy, w, "dy", shape, t, cur)
    hp, hs = _rows(h, w, "h", shape, t, cur)
    dp, ds = _rows(dh, w, "dh", shape, t, cur)
    xp, xs = _rows(dx, w, "dx", shape, t, cur)
    st = load_library().basp_rmsnorm_backward(
        code, shape[0], shape[1], yp, ys, hp, hs, _vector(rstd, w, "rstd", shape[0], _F32, cur),
        _vector(weight, w, "weight", shape[1], weight.dtype, cur), wcode, dp, ds, xp, xs,
        _vector(dweight, w, "dweight", shape[1], _F32, cur),
        _tptr(workspace, None, w, "workspace", "device", cur), _nbytes(workspace), _stream(stream))
    if st:
        _check(st, w)


def basp_layernorm(x, residual, weight, bias, eps, h=None, y=None, q=None, mean=None, rstd=None, stream=None):
    """Residual addition + layer norm; see ``basp_fp8.h``."""
    w = "basp_layernorm"
    shape, t = _2d(x, w, "x"), x.dtype
    code, wcode, cur = fp8_dtype_code(t), fp8_dtype_code(weight.dtype), _current_device()
    xp, xs = _rows(x, w, "x", shape, t, cur)
    rp, rs = _rows(residual, w, "residual", shape, t, cur)
    hp, hs = _rows(h, w, "h", shape, t, cur)
    yp, ys = _rows(y, w, "y", shape, t, cur)
    _check(load_library().basp_layernorm(
        code, shape[0], shape[1], xp, xs, rp, rs, _vector(weight, w, "weight", shape[1], weight.dtype, cur),
        _vector(bias, w, "bias", shape[1], weight.dtype, cur), wcode, eps, hp, hs, yp, ys, q,
        _vector(mean, w, "mean", shape[0], _F32, cur), _vector(rstd, w, "rstd", shape[0], _F32, cur),
        _stream(stream)), w)


def basp_layernorm_backward_workspace(rows: int, cols: int) -> int:
    return load_library().basp_layernorm_backward_workspace(rows, cols)


def basp_layernorm_backward(dy, h, mean, rstd, weight, dh, dx, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradient of :func:`basp_layernorm`; see ``basp_fp8.h``."""
    w = "basp_layernorm_backward"
    shape, t = _2d(dy, w, "dy"), dy.dtype
    code, wcode, cur = fp8_dtype_code(t), fp8_dtype_code(weight.dtype), _current_device()
    yp, ys = _rows(dy, w, "dy", shape, t, cur)
    hp, hs = _rows(h, w, "h", shape, t, cur)
    dp, ds = _rows(dh, w, "dh", shape, t, cur)
    xp, xs = _rows(dx, w, "dx", shape, t, cur)
    _check(load_library().basp_layernorm_backward(
        code, shape[0], shape[1], yp, ys, hp, hs, _vector(mean, w, "mean", shape[0], _F32, cur),
        _vector(rstd, w, "rstd", shape[0], _F32, cur), _vector(weight, w, "weight", shape[1], weight.dtype, cur),
        wcode, dp, ds, xp, xs, _vector(dweight, w, "dweight", shape[1], _F32, cur),
        _vector(dbias, w, "dbias", shape[1], _F32, cur), _tptr(workspace, None, w, "workspace", "device", cur),
        _nbytes(workspace), _stream(stream)), w)


def basp_quantize_fp8(x, q=None, qt=None, stream=None):
    """A matrix, and its transpose, to 8 bits; see ``basp_fp8.h``.  ``q`` and
    ``qt`` are :class:`basp_fp8_matrix` or None."""
    w = "basp_quantize_fp8"
    shape = _2d(x, w, "x")
    code = fp8_dtype_code(x.dtype)
    xp, xs = _rows(x, w, "x", shape, x.dtype, _current_device())
    st = load_library().basp_quantize_fp8(code, shape[0], shape[1], xp, xs, q, qt, _stream(stream))
    if st:
        _check(st, w)


def basp_matmul_fp8(a, b, bias, c, accumulate=False, stream=None):
    """C = A B^T (+ bias) (+ C); see ``basp_fp8.h``.  ``a`` and ``b`` are
    :class:`basp_fp8_matrix`."""
    w = "basp_matmul_fp8"
    t, n, cur = c.dtype, b.rows, _current_device()
    code = fp8_dtype_code(t)
    cp, cs = _rows(c, w, "c", (a.rows, n), t, cur)
    st = load_library().basp_matmul_fp8(a, b, _vector(bias, w, "bias", n, t, cur), int(accumulate), code, cp, cs,
                                        _stream(stream))
    if st:
        _check(st, w)


def fp8_entry_points():
    """Addresses of the loaded library's 8-bit entry points, in the order in
    which the torch module (``csrc/torch_ops.cpp``) takes them."""
    lib = load_library()
    return tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in FP8_EXPORTS[:5])


def layer_entry_points():
    """Addresses of the loaded library's other entry points that the torch module
    takes, in its order."""
    lib = load_library()
    return tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                 for n in FP8_EXPORTS[6:] + ATTENTION_EXPORTS[:5] + OPTIM_EXPORTS)


def basp_matmul_fp8_timeouts() -> int:
    """Read and clear the count of waits that ran out in the product's kernel
    on the current device (synchronises it)."""
    n = ctypes.c_ulonglong()
    _check(load_library().basp_matmul_fp8_timeouts(ctypes.byref(n)), "basp_matmul_fp8_timeouts")
    return n.value


# ---- attention and the optimiser (include/basp_attention.h, include/basp_optim.h) ----

# Their structures (basp_attention_desc, basp_heads, basp_adamw_tensor,
# basp_adamw_options) are filled by the caller; ``attention`` and ``optim`` have the
# calls on torch tensors.

def basp_attention(desc, q, k, v, o, lse=None, stream=None, o_rest=None):
    """Attention with a window and sinks; see ``basp_attention.h``."""
    _check(load_library().basp_attention(desc, q, k, v, o, o_rest, _ptr(lse), _stream(stream)), "basp_attention")


def basp_attention_backward_workspace(desc) -> int:
    return load_library().basp_attention_backward_workspace(desc)


def basp_attention_backward(desc, q, k, v, o, lse, d_o, dq, dk, dv, workspace, workspace_bytes=None, stream=None,
                            o_rest=None):
    """Gradients of :func:`basp_attention`; see ``basp_attention.h``."""
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check(load_library().basp_attention_backward(desc, q, k, v, o, o_rest, _ptr(lse), d_o, dq, dk, dv, _ptr(workspace),
                                                  wb, _stream(stream)), "basp_attention_backward")


def basp_attention_decode_workspace(desc) -> int:
    return load_library().basp_attention_decode_workspace(desc)


def basp_attention_decode(desc, q, k, v, lengths, o, workspace=None, workspace_bytes=None, stream=None):
    """One new token of each sequence over a cache; see ``basp_attention.h``."""
    wb = _nbytes(workspace) if workspace_bytes is None else workspace_bytes
    _check(load_library().basp_attention_decode(desc, q, k, v, _ptr(lengths), o, _ptr(workspace), wb,
                                                _stream(stream)), "basp_attention_decode")


def basp_attention_timeouts() -> int:
    """Read and clear the count of waits that ran out in the attention kernels on
    the current device (synchronises it)."""
    n = ctypes.c_ulonglong()
    _check(load_library().basp_attention_timeouts(ctypes.byref(n)), "basp_attention_timeouts")
    return n.value


def basp_adamw(tensors, options, stream=None):
    """A step of AdamW over a sequence of :class:`basp_adamw_tensor`; see
    ``basp_optim.h``."""
    table = (basp_adamw_tensor * len(tensors))(*tensors)
    _check(load_library().basp_adamw(table, len(tensors), options, _stream(stream)), "basp_adamw")


def basp_adamw_each(tensors, steps_at, options, stream=None, numbers=None):
    """The same with a number of steps for each tensor (int32 tensors or addresses on the
    GPU, or None), and with the tensors' numbers for the random bits."""
    w, n = "basp_adamw_each", len(tensors)
    for name, x in (("steps", steps_at), ("tensors", numbers)):
        if x is not None and len(x) != n:
            raise ValueError("%s: %d numbers of %s for %d tensors" % (w, len(x), name, n))
    at = None if steps_at is None else (ctypes.c_void_p * n)(*(_ptr(s) for s in steps_at))
    no = None if numbers is None else (ctypes.c_uint32 * n)(*numbers)
    _check(load_library().basp_adamw_each((basp_adamw_tensor * n)(*tensors), at, no, n, options, _stream(stream)), w)


class Layout:
    """Owns one layout handle; ``info`` holds the derived sizes."""

    def __init__(self, B, S, Hq, Hkv, d, N, K, dtype="bf16", order="bshd"):
        self.handle = basp_layout_create_ex(B, S, Hq, Hkv, d, N, K, dtype, order)
        self.info = basp_layout_query(self.handle)

    def close(self):
        if self.handle:
            basp_layout_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
