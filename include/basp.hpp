// basp.hpp -- header-only C++ convenience layer over the C ABI in basp.h.
//
// Adds nothing to what the C entry points do: basp::Layout owns a handle
// (destroyed with the object), exposes its basp_info, and forwards to the C
// calls, turning a non-OK status into a basp::Error that carries the status
// code.  All arguments, layouts and rules are those of basp.h.
#ifndef BASP_HPP
#define BASP_HPP

#include <stdexcept>
#include <string>
#include <utility>

#include "basp.h"
#include "basp_attention.h"
#include "basp_fp8.h"
#include "basp_optim.h"

namespace basp {

class Error : public std::runtime_error {
public:
    Error(basp_status status, const char *where)
        : std::runtime_error(std::string(where) + ": " + basp_status_string(status)),
          status_(status) {}
    basp_status status() const { return status_; }

private:
    basp_status status_;
};

inline void check(basp_status s, const char *where) {
    if (s != BASP_OK) throw Error(s, where);
}

class Layout {
public:
    // K = 0 asks for the BASP rule K = N / B.
    Layout(int64_t B, int64_t S, int64_t Hq, int64_t Hkv, int64_t d, int64_t N,
           int64_t K, basp_dtype dtype = BASP_DTYPE_BF16,
           basp_order order = BASP_ORDER_BSHD) {
        const basp_layout_desc desc = {B, S, Hq, Hkv, d, N, K, dtype, order};
        check(basp_layout_create_ex(&desc, &handle_), "basp_layout_create_ex");
        check(basp_layout_query(handle_, &info_), "basp_layout_query");
    }
    ~Layout() { basp_layout_destroy(handle_); }
    Layout(const Layout &) = delete;
    Layout &operator=(const Layout &) = delete;
    Layout(Layout &&o) noexcept : handle_(o.handle_), info_(o.info_) { o.handle_ = nullptr; }
    Layout &operator=(Layout &&o) noexcept {
        std::swap(handle_, o.handle_);
        std::swap(info_, o.info_);
        return *this;
    }

    const basp_layout *handle() const { return handle_; }
    const basp_info &info() const { return info_; }

    // seq-sharded -> head-sharded (any of the three pairs may be null)
    void seq2head(const void *q, const void *k, const void *v, void *q_out,
                  void *k_out, void *v_out, cudaStream_t stream,
                  basp_algo algo = BASP_ALGO_FUSED, void *workspace = nullptr,
                  size_t workspace_bytes = 0) const {
        check(basp_seq2head(handle_, algo, q, k, v, q_out, k_out, v_out, workspace,
                            workspace_bytes, stream), "basp_seq2head");
    }
    // head-sharded -> seq-sharded
    void head2seq(const void *o, const void *k, const void *v, void *o_out,
                  void *k_out, void *v_out, cudaStream_t stream,
                  basp_algo algo = BASP_ALGO_FUSED, void *workspace = nullptr,
                  size_t workspace_bytes = 0) const {
        check(basp_head2seq(handle_, algo, o, k, v, o_out, k_out, v_out, workspace,
                            workspace_bytes, stream), "basp_head2seq");
    }
    // packed QKV projection output -> head-sharded Q, K, V, and back
    void seq2head_qkv(const void *qkv, void *q_out, void *k_out, void *v_out,
                      cudaStream_t stream) const {
        check(basp_seq2head_qkv(handle_, qkv, q_out, k_out, v_out, stream),
              "basp_seq2head_qkv");
    }
    void head2seq_qkv(const void *q, const void *k, const void *v, void *qkv_out,
                      cudaStream_t stream) const {
        check(basp_head2seq_qkv(handle_, q, k, v, qkv_out, stream), "basp_head2seq_qkv");
    }
    // host buffers in and out: staged through caller-owned device `staging`,
    // or (staging null) read and written in place when page-locked
    void seq2head_host(const void *q, const void *k, const void *v, void *q_out,
                       void *k_out, void *v_out, void *staging, size_t staging_bytes,
                       cudaStream_t stream, basp_algo algo = BASP_ALGO_FUSED,
                       void *workspace = nullptr, size_t workspace_bytes = 0) const {
        check(basp_seq2head_host(handle_, algo, q, k, v, q_out, k_out, v_out, staging,
                                 staging_bytes, workspace, workspace_bytes, stream),
              "basp_seq2head_host");
    }
    void head2seq_host(const void *o, const void *k, const void *v, void *o_out,
                       void *k_out, void *v_out, void *staging, size_t staging_bytes,
                       cudaStream_t stream, basp_algo algo = BASP_ALGO_FUSED,
                       void *workspace = nullptr, size_t workspace_bytes = 0) const {
        check(basp_head2seq_host(handle_, algo, o, k, v, o_out, k_out, v_out, staging,
                                 staging_bytes, workspace, workspace_bytes, stream),
              "basp_head2seq_host");
    }

private:
    basp_layout *handle_ = nullptr;
    basp_info info_{};
};

// ---- the 8-bit projections (basp_fp8.h): the same calls, throwing ------------

inline void rmsnorm(basp_dtype dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                    const void *residual, int64_t residual_stride, const void *weight,
                    basp_dtype weight_dtype, float eps, void *h, int64_t h_stride, void *y,
                    int64_t y_stride, const basp_fp8_matrix *q, float *rstd, cudaStream_t stream) {
    check(basp_rmsnorm(dtype, rows, cols, x, x_stride, residual, residual_stride, weight, weight_dtype,
                       eps, h, h_stride, y, y_stride, q, rstd, stream), "basp_rmsnorm");
}
inline void rmsnorm_backward(basp_dtype dtype, int64_t rows, int64_t cols, const void *dy,
                             int64_t dy_stride, const void *h, int64_t h_stride, const float *rstd,
                             const void *weight, basp_dtype weight_dtype, const void *dh,
                             int64_t dh_stride, void *dx, int64_t dx_stride, float *dweight,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    check(basp_rmsnorm_backward(dtype, rows, cols, dy, dy_stride, h, h_stride, rstd, weight,
                                weight_dtype, dh, dh_stride, dx, dx_stride, dweight, workspace,
                                workspace_bytes, stream), "basp_rmsnorm_backward");
}
inline void quantize_fp8(basp_dtype dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                         const basp_fp8_matrix *q, const basp_fp8_matrix *qt, cudaStream_t stream) {
    check(basp_quantize_fp8(dtype, rows, cols, x, x_stride, q, qt, stream), "basp_quantize_fp8");
}
inline void matmul_fp8(const basp_fp8_matrix &a, const basp_fp8_matrix &b, const void *bias,
                       bool accumulate, basp_dtype dtype, void *c, int64_t c_stride,
                       cudaStream_t stream) {
    check(basp_matmul_fp8(&a, &b, bias, accumulate, dtype, c, c_stride, stream), "basp_matmul_fp8");
}

inline void layernorm(basp_dtype dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride,
                      const void *residual, int64_t residual_stride, const void *weight, const void *bias,
                      basp_dtype weight_dtype, float eps, void *h, int64_t h_stride, void *y, int64_t y_stride,
                      const basp_fp8_matrix *q, float *mean, float *rstd, cudaStream_t stream) {
    check(basp_layernorm(dtype, rows, cols, x, x_stride, residual, residual_stride, weight, bias, weight_dtype,
                         eps, h, h_stride, y, y_stride, q, mean, rstd, stream), "basp_layernorm");
}
inline void layernorm_backward(basp_dtype dtype, int64_t rows, int64_t cols, const void *dy, int64_t dy_stride,
                               const void *h, int64_t h_stride, const float *mean, const float *rstd,
                               const void *weight, basp_dtype weight_dtype, const void *dh, int64_t dh_stride,
                               void *dx, int64_t dx_stride, float *dweight, float *dbias, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    check(basp_layernorm_backward(dtype, rows, cols, dy, dy_stride, h, h_stride, mean, rstd, weight,
                                  weight_dtype, dh, dh_stride, dx, dx_stride, dweight, dbias, workspace,
                                  workspace_bytes, stream), "basp_layernorm_backward");
}

// ---- attention (basp_attention.h) and the optimiser's step (basp_optim.h) ------

inline void attention(const basp_attention_desc &desc, const basp_heads &q, const basp_heads &k,
                      const basp_heads &v, const basp_heads &o, float *lse, cudaStream_t stream,
                      const basp_heads *o_rest = nullptr) {
    check(basp_attention(&desc, &q, &k, &v, &o, o_rest, lse, stream), "basp_attention");
}
inline void attention_backward(const basp_attention_desc &desc, const basp_heads &q, const basp_heads &k,
                               const basp_heads &v, const basp_heads &o, const float *lse,
                               const basp_heads &d_o, const basp_heads &dq, const basp_heads &dk,
                               const basp_heads &dv, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream, const basp_heads *o_rest = nullptr) {
    check(basp_attention_backward(&desc, &q, &k, &v, &o, o_rest, lse, &d_o, &dq, &dk, &dv, workspace, workspace_bytes,
                                  stream), "basp_attention_backward");
}
inline void attention_decode(const basp_attention_desc &desc, const basp_heads &q, const basp_heads &k,
                             const basp_heads &v, const int32_t *lengths, const basp_heads &o, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
    check(basp_attention_decode(&desc, &q, &k, &v, lengths, &o, workspace, workspace_bytes, stream),
          "basp_attention_decode");
}
inline void adamw(const basp_adamw_tensor *tensors, int64_t count, const basp_adamw_options &options,
                  cudaStream_t stream) {
    check(basp_adamw(tensors, count, &options, stream), "basp_adamw");
}
inline void adamw_each(const basp_adamw_tensor *tensors, const int32_t *const *steps_at, const uint32_t *numbers,
                       int64_t count, const basp_adamw_options &options, cudaStream_t stream) {
    check(basp_adamw_each(tensors, steps_at, numbers, count, &options, stream), "basp_adamw_each");
}

}  // namespace basp

#endif  // BASP_HPP
