// norm_common.cuh -- what the norms' forward and backward kernels share: sums over
// a row, roots, and the choice of a kernel's types.
#pragma once

#include "fp8_common.cuh"

namespace basp_fp8 {

// 1 / sqrt(x) to half a unit in the last place: the hardware's estimate and
// one Newton step on the residual 1 - x r^2, taken exactly.  (A value next to
// a border of two 8-bit values is decided by this last bit.)
__device__ __forceinline__ float inverse_root(float x) {
    const float r = rsqrtf(x);
    const float t = x * r;
    const float e = fmaf(-t, r, 1.f) - fmaf(x, r, -t) * r;
    const float better = fmaf(0.5f * r, e, r);
    return better == better ? better : r;                // x = 0 or infinite: the estimate says it
}

// sum / n to half a unit in the last place, given 1 / n.
__device__ __forceinline__ float mean_of(float sum, float n, float inv_n) {
    const float q = sum * inv_n;
    const float better = fmaf(fmaf(-q, n, sum), inv_n, q);
    return better == better ? better : q;                // an infinite sum
}

// Sum over the warps of one row: warps of a row are blockDim.x / 32, rows of
// a CTA blockDim.y (more than one only with one warp a row).
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum over all warps of the CTA's row, the same in every thread: every
// warp adds the warps' parts in the same order.
__device__ __forceinline__ float row_sum(float v, float *part, int warps) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.f;
    return warp_sum(v);
}

// ---- rows on their way to shared memory ----------------------------------------

constexpr int kAhead = 2;            // rows ahead of the one that is worked on
constexpr int kWalkThreads = 512;    // threads of a CTA that walks rows, at most

// As row_sum, for whole rows a CTA and with fewer instructions: every thread
// adds the warps' parts itself.  `part` has room for 16 and is zero past the
// CTA's warps.
__device__ __forceinline__ float walk_sum(float v, float *part, int warps) {
    v = warp_sum(v);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; i += 4) {
        const float4 p = *reinterpret_cast<const float4 *>(part + i);
        v += (p.x + p.y) + (p.z + p.w);
    }
    return v;
}

// Largest over the threads of a 128-block (16 or 32 of a warp).
template <int THREADS> __device__ __forceinline__ uint32_t block_max(uint32_t m) {
    if constexpr (THREADS == 32) {
        return __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
        for (int o = THREADS / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    }
}

// Calls f<T, W, VEC>() for the run-time types.
template <class F>
inline basp_status dispatch(basp_dtype t, basp_dtype w, bool vec, F &&f) {
    auto with = [&](auto te, auto we) {
        return vec ? f(te, we, std::true_type()) : f(te, we, std::false_type());
    };
    if (t == BASP_DTYPE_FP32) return with(float(), float());
    if (t == BASP_DTYPE_BF16)
        return w == BASP_DTYPE_FP32 ? with(__nv_bfloat16(), float()) : with(__nv_bfloat16(), __nv_bfloat16());
    return w == BASP_DTYPE_FP32 ? with(__half(), float()) : with(__half(), __half());
}

}  // namespace basp_fp8
