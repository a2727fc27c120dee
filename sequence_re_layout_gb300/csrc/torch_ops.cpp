// torch_ops.cpp -- the 8-bit operators on torch tensors: checks of arguments,
// outputs, and the C calls of basp_fp8.h, as a CPython module without pybind.
// fp8.py is its only user.  It is compiled code because the calls are short: a
// token's norm takes two microseconds on the GPU, its four outputs and the
// checks took twenty in Python.
//
// Every function runs on the current device's current stream, on which torch's
// allocator hands out the outputs.  A wrong argument is a ValueError before
// anything is launched; a status of the C call is a BaspError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <optional>
#include <sstream>
#include <string>

#include "basp_fp8.h"

namespace {

using at::Tensor;

constexpr int64_t kBlock = BASP_FP8_BLOCK;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

PyObject *g_error = nullptr;               // the binding's BaspError

// The entry points of the library that the binding has loaded (there are
// several builds of it).
struct Library {
    decltype(&basp_rmsnorm) rmsnorm;
    decltype(&basp_rmsnorm_backward) rmsnorm_backward;
    decltype(&basp_rmsnorm_backward_workspace) rmsnorm_backward_workspace;
    decltype(&basp_quantize_fp8) quantize;
    decltype(&basp_matmul_fp8) matmul;
} g_lib;

[[noreturn]] void refuse(const char *where, const std::string &what) {
    throw c10::ValueError({__func__, __FILE__, uint32_t(__LINE__)}, std::string(where) + ": " + what);
}

template <class... A> std::string text(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    return s.str();
}

const Tensor *tensor(PyObject *o, const char *where, const char *name, bool may_be_none = false) {
    if (o == Py_None && may_be_none) return nullptr;
    if (!THPVariable_Check(o)) refuse(where, text(name, " must be a tensor"));
    return &THPVariable_Unpack(o);
}

basp_dtype dtype_code(at::ScalarType t, const char *where, const char *name) {
    switch (t) {
        case at::kBFloat16: return BASP_DTYPE_BF16;
        case at::kHalf: return BASP_DTYPE_FP16;
        case at::kFloat: return BASP_DTYPE_FP32;
        default: refuse(where, text(name, " must be bfloat16, float16 or float32, got ", c10::toString(t)));
    }
}

void on_device(const Tensor &x, int device, const char *where, const char *name) {
    if (!x.is_cuda() || x.get_device() != device)
        refuse(where, text(name, " must be on the current device cuda:", device, ", it is on ", x.device().str()));
}

// New tensors on the GPU, straight from the allocator: at::empty goes through
// the dispatcher first (a token's norm, of four tensors: 9.3 us of host time so,
// 7.4 now).
Tensor new_tensor(c10::IntArrayRef sizes, at::ScalarType type, c10::Device device) {
    return Tensor(at::detail::empty_cuda(sizes, type, device, std::nullopt));
}

// A caller's tensor that a call will write to.  The calls are no operations of
// autograd, so one whose gradient autograd would follow is refused, as torch
// refuses it for an out=; `written` tells autograd of the write, so that a tensor
// that was saved for a backward pass and overwritten is noticed there.
void may_write(const Tensor *t, const char *where, const char *name) {
    if (t != nullptr && c10::GradMode::is_enabled() && t->requires_grad())
        refuse(where, text(name, " is written to and must not require a gradient (outside of no_grad)"));
}
void written(const Tensor *t) {
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// A matrix of [rows][cols] as the C calls take it.
struct Rows {
    void *p = nullptr;
    int64_t stride = 0;
};

// x [..., cols] as rows x cols; leading dimensions have to lie as one.
Rows rows_of(const Tensor *x, int64_t rows, int64_t cols, at::ScalarType type, int device, const char *where,
             const char *name) {
    Rows r;
    if (x == nullptr) return r;
    on_device(*x, device, where, name);
    if (x->scalar_type() != type)
        refuse(where, text(name, " must be ", c10::toString(type), ", got ", c10::toString(x->scalar_type())));
    const int64_t d = x->dim();
    if (d < 1 || x->size(-1) != cols || x->numel() != rows * cols)
        refuse(where, text(name, " must have ", rows, " rows of ", cols, ", got shape ", x->sizes()));
    if (rows == 0 || cols == 0) return r;
    if (cols > 1 && x->stride(-1) != 1)
        refuse(where, text(name, " must have its columns next to each other, got strides ", x->strides()));
    r.p = x->data_ptr();
    r.stride = cols;                                      // of a single row it says nothing
    int64_t span = -1;                                    // stride of the next dimension outwards
    for (int64_t i = d - 2; i >= 0; --i) {
        if (x->size(i) == 1) continue;
        if (span < 0) r.stride = x->stride(i);
        else if (x->stride(i) != span)
            refuse(where, text("the rows of ", name, " must lie evenly, got shape ", x->sizes(), " and strides ",
                               x->strides()));
        span = x->stride(i) * x->size(i);
    }
    return r;
}

void *vector_of(const Tensor *x, int64_t n, at::ScalarType type, int device, const char *where, const char *name) {
    if (x == nullptr) return nullptr;
    on_device(*x, device, where, name);
    if (x->scalar_type() != type)
        refuse(where, text(name, " must be ", c10::toString(type), ", got ", c10::toString(x->scalar_type())));
    if (x->dim() != 1 || x->size(0) != n || (n > 1 && x->stride(0) != 1))
        refuse(where, text(name, " must be a contiguous vector of ", n, ", got shape ", x->sizes()));
    return n > 0 ? x->data_ptr() : nullptr;
}

// ---- 8-bit matrices ---------------------------------------------------------

struct Fp8 {
    Tensor data, scales;
    basp_fp8_matrix c = {};
};

Fp8 new_fp8(int64_t rows, int64_t cols, int64_t block_rows, const c10::Device &device) {
    const int64_t blocks = ceil_div(cols, kBlock), srows = ceil_div(rows, block_rows);
    // A product reads rows in pieces of 128 bytes: 1021 x 2999 x 1543 takes 10.6
    // us where those are whole cache lines, 11.0 where they are not.
    const int64_t pitch = round_up(cols, cols > 128 ? 128 : 16), spitch = round_up(blocks, 4);
    Fp8 f;
    f.data = Tensor(at::detail::empty_strided_cuda({rows, cols}, {pitch, 1}, at::kFloat8_e4m3fn, device));
    f.scales = Tensor(at::detail::empty_strided_cuda({srows, blocks}, {spitch, 1}, at::kFloat8_e8m0fnu, device));
    f.c = {f.data.data_ptr(), f.scales.data_ptr(), rows, cols, pitch, spitch, block_rows};
    return f;
}

basp_fp8_matrix fp8_of(PyObject *od, PyObject *os, int64_t block_rows, int device, const char *where,
                       const char *name) {
    const Tensor &d = *tensor(od, where, name), &s = *tensor(os, where, name);
    on_device(d, device, where, name);
    on_device(s, device, where, name);
    if (d.scalar_type() != at::kFloat8_e4m3fn || s.scalar_type() != at::kFloat8_e8m0fnu)
        refuse(where, text(name, " must be float8_e4m3fn with scales of float8_e8m0fnu, got ",
                           c10::toString(d.scalar_type()), " and ", c10::toString(s.scalar_type())));
    if (block_rows != 1 && block_rows != kBlock)
        refuse(where, text("block_rows of ", name, " must be 1 or ", kBlock, ", got ", block_rows));
    if (d.dim() != 2 || s.dim() != 2) refuse(where, text(name, " must have two dimensions"));
    const int64_t rows = d.size(0), cols = d.size(1), srows = ceil_div(rows, block_rows);
    const int64_t blocks = ceil_div(cols, kBlock);
    if (s.size(0) != srows || s.size(1) != blocks)
        refuse(where, text("scales of shape ", s.sizes(), " do not fit ", name, " of shape ", d.sizes(),
                           " with block_rows ", block_rows));
    if ((cols > 1 && d.stride(1) != 1) || (blocks > 1 && s.stride(1) != 1))
        refuse(where, text("columns of ", name, " must be next to each other"));
    // the stride of a single row says nothing: one that the C call accepts
    return {d.data_ptr(), s.data_ptr(), rows, cols, rows > 1 ? d.stride(0) : round_up(cols, 16),
            srows > 1 ? s.stride(0) : round_up(blocks, 4), block_rows};
}

// ---- Python ---------------------------------------------------------------------

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }

PyObject *wrap_or_none(const Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

template <class... P> PyObject *tuple(P... items) {
    PyObject *const all[] = {items...};
    constexpr Py_ssize_t n = sizeof...(P);
    PyObject *t = PyTuple_New(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (t != nullptr && all[i] != nullptr) PyTuple_SET_ITEM(t, i, all[i]);
        else Py_XDECREF(all[i]);
    }
    return t;
}

// Raises BaspError(status, where) and returns false unless the status is OK.
bool check(basp_status st, const char *where) {
    if (st == BASP_OK) return true;
    PyObject *e = PyObject_CallFunction(g_error, "is", int(st), where);
    if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}

bool arguments(Py_ssize_t got, Py_ssize_t want, const char *where) {
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", where, want, got);
    return false;
}

struct Call {
    int device = -1;
    cudaStream_t stream = nullptr;
    Call(const Tensor &x, const char *where, const char *name) {
        if (!x.is_cuda()) refuse(where, text(name, " must be on a CUDA device, it is on ", x.device().str()));
        device = c10::cuda::current_device();
        stream = c10::cuda::getCurrentCUDAStream(device).stream();
    }
};

// The rows and columns of x [..., cols].
void sides(const Tensor &x, const char *where, const char *name, int64_t *rows, int64_t *cols) {
    if (x.dim() < 1) refuse(where, text(name, " must have at least one dimension"));
    *cols = x.size(-1);
    *rows = 1;
    for (int64_t i = 0; i + 1 < x.dim(); ++i) *rows *= x.size(i);
}

// rmsnorm(x, weight, residual, eps, quantized, h) -> (y or data, scales or None, h or None, rstd)
PyObject *rmsnorm(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char *where = "rmsnorm";
    if (!arguments(n, 6, where)) return nullptr;
    const Tensor &x = *tensor(args[0], where, "x"), &weight = *tensor(args[1], where, "weight");
    const Tensor *residual = tensor(args[2], where, "residual", true);
    const double eps = PyFloat_AsDouble(args[3]);
    if (PyErr_Occurred()) return nullptr;
    const bool quantized = args[4] == Py_True;
    const Tensor *given = tensor(args[5], where, "h", true);
    may_write(given, where, "h");
    const auto type = x.scalar_type();
    const basp_dtype code = dtype_code(type, where, "x"), wcode = dtype_code(weight.scalar_type(), where, "weight");
    int64_t rows, cols;
    sides(x, where, "x", &rows, &cols);
    const Call call(x, where, "x");
    const Rows rx = rows_of(&x, rows, cols, type, call.device, where, "x");
    const Rows rr = rows_of(residual, rows, cols, type, call.device, where, "residual");
    const void *w = vector_of(&weight, cols, weight.scalar_type(), call.device, where, "weight");
    Tensor h;
    if (given != nullptr) h = *given;
    else if (residual != nullptr) h = new_tensor(x.sizes(), type, x.device());
    const Rows rh = rows_of(h.defined() ? &h : nullptr, rows, cols, type, call.device, where, "h");
    const Tensor rstd = new_tensor({rows}, at::kFloat, x.device());
    Fp8 q;
    Tensor y;
    Rows ry;
    if (quantized) {
        q = new_fp8(rows, cols, 1, x.device());
    } else {
        y = new_tensor(x.sizes(), type, x.device());
        ry = rows_of(&y, rows, cols, type, call.device, where, "y");
    }
    // the C call wants one of y and q even where there is nothing to write; the
    // mean of no columns is 0 / 0
    if (cols == 0) rstd.fill_(std::numeric_limits<double>::quiet_NaN());
    if (rows > 0 && cols > 0 &&
        !check(g_lib.rmsnorm(code, rows, cols, rx.p, rx.stride, rr.p, rr.stride, w, wcode, float(eps), rh.p, rh.stride,
                            ry.p, ry.stride, quantized ? &q.c : nullptr, rstd.data_ptr<float>(), call.stream),
               "basp_rmsnorm"))
        return nullptr;
    written(given);
    return tuple(wrap(quantized ? q.data : y), wrap_or_none(q.scales), wrap_or_none(h), wrap(rstd));
    END_HANDLE_TH_ERRORS
}

// rmsnorm_backward(dy, h, rstd, weight, dh, need_dweight) -> (dx, dweight or None)
PyObject *rmsnorm_backward(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char *where = "rmsnorm_backward";
    if (!arguments(n, 6, where)) return nullptr;
    const Tensor &dy = *tensor(args[0], where, "dy"), &h = *tensor(args[1], where, "h");
    const Tensor &rstd = *tensor(args[2], where, "rstd"), &weight = *tensor(args[3], where, "weight");
    const Tensor *dh = tensor(args[4], where, "dh", true);
    const bool need = args[5] == Py_True;
    const auto type = dy.scalar_type();
    const basp_dtype code = dtype_code(type, where, "dy"), wcode = dtype_code(weight.scalar_type(), where, "weight");
    int64_t rows, cols;
    sides(dy, where, "dy", &rows, &cols);
    const Call call(dy, where, "dy");
    const Rows ry = rows_of(&dy, rows, cols, type, call.device, where, "dy");
    const Rows rh = rows_of(&h, rows, cols, type, call.device, where, "h");
    const Rows rd = rows_of(dh, rows, cols, type, call.device, where, "dh");
    const void *r = vector_of(&rstd, rows, at::kFloat, call.device, where, "rstd");
    const void *w = vector_of(&weight, cols, weight.scalar_type(), call.device, where, "weight");
    const Tensor dx = new_tensor(dy.sizes(), dy.scalar_type(), dy.device());
    const Rows rx = rows_of(&dx, rows, cols, type, call.device, where, "dx");
    Tensor dweight, workspace;
    const int64_t bytes = need ? g_lib.rmsnorm_backward_workspace(rows, cols) : 0;
    if (need) {
        dweight = new_tensor({cols}, at::kFloat, dy.device());
        workspace = new_tensor({bytes}, at::kByte, dy.device());
    }
    if (!check(g_lib.rmsnorm_backward(code, rows, cols, ry.p, ry.stride, rh.p, rh.stride, static_cast<const float *>(r),
                                     w, wcode, rd.p, rd.stride, rx.p, rx.stride,
                                     need && cols > 0 ? dweight.data_ptr<float>() : nullptr,
                                     bytes > 0 ? workspace.data_ptr() : nullptr, size_t(bytes), call.stream),
               "basp_rmsnorm_backward"))
        return nullptr;
    return tuple(wrap(dx), wrap_or_none(dweight));
    END_HANDLE_TH_ERRORS
}

// quantize(x, block_rows, rows, transposed) -> (data, scales, data of the transpose, its scales), None where not asked
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char *where = "quantize";
    if (!arguments(n, 4, where)) return nullptr;
    const Tensor &x = *tensor(args[0], where, "x");
    const int64_t block_rows = PyLong_AsLongLong(args[1]);
    if (PyErr_Occurred()) return nullptr;
    const bool want = args[2] == Py_True, want_t = args[3] == Py_True;
    if (block_rows != 1 && block_rows != kBlock)
        refuse(where, text("block_rows must be 1 or ", kBlock, ", got ", block_rows));
    if (!want && !want_t) refuse(where, "nothing asked for: neither rows nor transposed");
    const basp_dtype code = dtype_code(x.scalar_type(), where, "x");
    int64_t rows, cols;
    sides(x, where, "x", &rows, &cols);
    const Call call(x, where, "x");
    const Rows rx = rows_of(&x, rows, cols, x.scalar_type(), call.device, where, "x");
    Fp8 q, qt;
    if (want) q = new_fp8(rows, cols, block_rows, x.device());
    if (want_t) qt = new_fp8(cols, rows, block_rows, x.device());
    if (!check(g_lib.quantize(code, rows, cols, rx.p, rx.stride, want ? &q.c : nullptr, want_t ? &qt.c : nullptr,
                                 call.stream), "basp_quantize_fp8"))
        return nullptr;
    return tuple(wrap_or_none(q.data), wrap_or_none(q.scales), wrap_or_none(qt.data), wrap_or_none(qt.scales));
    END_HANDLE_TH_ERRORS
}

// matmul(a, a_scales, a_block_rows, b, b_scales, b_block_rows, bias, out, out_dtype, accumulate) -> out
PyObject *matmul(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const char *where = "matmul";
    if (!arguments(n, 10, where)) return nullptr;
    const int64_t ab = PyLong_AsLongLong(args[2]), bb = PyLong_AsLongLong(args[5]);
    if (PyErr_Occurred()) return nullptr;
    const Call call(*tensor(args[0], where, "a"), where, "a");
    const basp_fp8_matrix a = fp8_of(args[0], args[1], ab, call.device, where, "a");
    const basp_fp8_matrix b = fp8_of(args[3], args[4], bb, call.device, where, "b");
    if (a.cols != b.cols) refuse(where, text("a has ", a.cols, " columns and b ", b.cols));
    const Tensor *bias = tensor(args[6], where, "bias", true), *given = tensor(args[7], where, "out", true);
    may_write(given, where, "out");
    const bool accumulate = args[9] == Py_True;
    if (accumulate && given == nullptr) refuse(where, "accumulate needs out");
    if (given == nullptr && !THPDtype_Check(args[8])) refuse(where, "out_dtype must be a torch.dtype");
    const auto type =
        given != nullptr ? given->scalar_type() : reinterpret_cast<THPDtype *>(args[8])->scalar_type;
    const basp_dtype code = dtype_code(type, where, "out");
    if (given != nullptr && given->dim() != 2) refuse(where, text("out must have two dimensions, got shape ", given->sizes()));
    const Tensor out = given != nullptr ? *given
                                        : new_tensor({a.rows, b.rows}, type, THPVariable_Unpack(args[0]).device());
    const Rows c = rows_of(&out, a.rows, b.rows, type, call.device, where, "out");
    if (given != nullptr && (given->size(0) != a.rows || given->size(1) != b.rows))
        refuse(where, text("out must have shape [", a.rows, ", ", b.rows, "], got ", given->sizes()));
    const void *bp = vector_of(bias, b.rows, type, call.device, where, "bias");
    if (!check(g_lib.matmul(&a, &b, bp, accumulate, code, c.p, c.stride, call.stream), "basp_matmul_fp8"))
        return nullptr;
    written(given);
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef g_methods[] = {
    {"rmsnorm", fast<rmsnorm>(), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", fast<rmsnorm_backward>(), METH_FASTCALL, nullptr},
    {"quantize", fast<quantize>(), METH_FASTCALL, nullptr},
    {"matmul", fast<matmul>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops() {
    PyObject *binding = PyImport_ImportModule("sequence_re_layout_gb300.binding");
    if (binding == nullptr) return nullptr;
    g_error = PyObject_GetAttrString(binding, "BaspError");
    PyObject *at = g_error != nullptr ? PyObject_CallMethod(binding, "fp8_entry_points", nullptr) : nullptr;
    Py_DECREF(binding);
    unsigned long long p[5];
    const bool ok = at != nullptr && PyArg_ParseTuple(at, "KKKKK", &p[0], &p[1], &p[2], &p[3], &p[4]);
    Py_XDECREF(at);
    if (!ok) return nullptr;
    g_lib.rmsnorm = reinterpret_cast<decltype(g_lib.rmsnorm)>(p[0]);
    g_lib.rmsnorm_backward = reinterpret_cast<decltype(g_lib.rmsnorm_backward)>(p[1]);
    g_lib.rmsnorm_backward_workspace = reinterpret_cast<decltype(g_lib.rmsnorm_backward_workspace)>(p[2]);
    g_lib.quantize = reinterpret_cast<decltype(g_lib.quantize)>(p[3]);
    g_lib.matmul = reinterpret_cast<decltype(g_lib.matmul)>(p[4]);
    return PyModule_Create(&g_module);
}
