// matvec.cuh -- basp_matmul_fp8 for up to eight tokens and a B of ordinary size.
//
// A tile of matmul.cu would be nearly all padding, and what surrounds it (the
// barriers, tensor memory, the join of a split K) takes longer than B takes to
// read.  Here a warp reads 16 rows of B straight into the registers that
// mma.sync wants, the tokens as its 8 columns; the warps of a CTA share K, and
// their sums are added in the warps' order.  One matrix instruction takes 32
// values of K; the sum over a block of 128 is scaled in 32 bits.
//
// What bounds it: latency (a launch, one trip to memory, one join: 2.4 us at
// 2048 x 2048), then mma.sync, which the counters show on the half-precision pipe,
// so that e4m3 operands are converted first; past some 16 million values of B it
// takes longer than reading them (131072 x 2048: 50 us, 42 on tcgen05).  In 80
// registers a thread 24 warps fit an SM (64 registers: 1 us more at 6144 x 2048).
#pragma once

#include "fp8_common.cuh"
#include "matmul_plan.h"

namespace basp_fp8 {

constexpr int kVecRows = 16;              // rows of B a warp
constexpr int kVecBlocks = 2;             // blocks of 128 along K that a warp is worth

struct MatvecArgs {
    const uint8_t *x, *w, *sx, *sw;       // A and B, and their scales
    int64_t x_pitch, w_pitch, sx_pitch, sw_pitch;
    int sx_shift, sw_shift;               // row -> scale row: 0 or 7
    void *c;
    const void *bias;
    int64_t c_stride;
    int M, N, K;
    int accumulate;
};

// 16 values of a row's last block, those past the first `left` zero.  The last
// ones are read one by one: what follows them may not be the matrix'.
__device__ __forceinline__ uint4 load_last(const uint8_t *p, int left) {
    if (left >= 16) return *reinterpret_cast<const uint4 *>(p);
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int j = left - 1; j >= 0; --j) {
        hi = hi << 8 | lo >> 56;
        lo = lo << 8 | p[j];
    }
    return make_uint4(uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32));
}

// c += a b of 16 rows of B's side, 32 values of K and 8 tokens.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 64 values of K: the order within them is free, and the same on both sides.
__device__ __forceinline__ void multiply64(float (&c)[4], const uint4 &p, const uint4 &q, const uint4 &x) {
    mma_e4m3(c, p.x, q.x, p.y, q.y, x.x, x.y);
    mma_e4m3(c, p.z, q.z, p.w, q.w, x.z, x.w);
}
// The products of the block that K ends in, `left` values from this lane's on.
// Not inlined: the registers are for the other blocks.
__device__ __noinline__ float4 multiply_last(const uint8_t *p, const uint8_t *q, const uint8_t *x, int left,
                                             bool token) {
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int k = 0; k < kBlock; k += 64, left -= 64) {
        const uint4 xv = load_last(x + k, token ? left : 0);
        multiply64(c, load_last(p + k, left), load_last(q + k, left), xv);
    }
    return make_float4(c[0], c[1], c[2], c[3]);
}

// v * 2^(ea + eb - 254) for two scale bytes; 255 is NaN.
__device__ __forceinline__ float scaled(float v, uint32_t ea, uint32_t eb) {
    const int e = int(ea + eb) - 127;                     // the product's biased exponent
    if (e > 0 && e < 255 && max(ea, eb) < 255u) return v * __uint_as_float(uint32_t(e) << 23);
    if (max(ea, eb) == 255u) return __uint_as_float(0x7fffffffu);
    // out of a float's range: half the power at a time
    const int half = (e - 127) / 2, rest = e - 127 - half;
    return v * __uint_as_float(uint32_t(half + 127) << 23) * __uint_as_float(uint32_t(rest + 127) << 23);
}

// W: the most warps of a CTA.  With eight, three CTAs fit an SM.
template <class T, int W>
__global__ void __launch_bounds__(W * 32, W > 8 ? 1 : 3) matvec_kernel(const __grid_constant__ MatvecArgs a) {
    __shared__ float4 part[W][32];
    grid_dependency();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane / 4, t = lane % 4;                 // fragments: rows g and g + 8, token g, 16 bytes t of 64
    const int warps = blockDim.x / 32;                    // each takes a part of K
    const int64_t n0 = int64_t(blockIdx.x) * kVecRows;
    const int blocks = (a.K - 1) / kBlock + 1;
    const int b0 = int(int64_t(blocks) * warp / warps), b1 = int(int64_t(blocks) * (warp + 1) / warps);

    // rows past the end: the last one's, and not stored; tokens: zeros
    const uint8_t *w[2], *sw[2], *sx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t n = min(n0 + g + 8 * i, int64_t(a.N) - 1), m = min(2 * t + i, a.M - 1);
        w[i] = a.w + n * a.w_pitch + 16 * t;
        sw[i] = a.sw + (n >> a.sw_shift) * a.sw_pitch;
        sx[i] = a.sx + (m >> a.sx_shift) * a.sx_pitch;
    }
    const bool token = g < a.M;
    const uint8_t *x = a.x + (token ? g : 0) * a.x_pitch + 16 * t;

    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int whole = min(b1, a.K / kBlock);
    for (int b = b0; b < whole; ++b) {
        const int64_t k = int64_t(b) * kBlock;
        uint4 wv[2][2], xv[2];                            // [64 values][row]
        uint32_t we[2], xe[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 2; ++i) wv[h][i] = *reinterpret_cast<const uint4 *>(w[i] + k + 64 * h);
            xv[h] = token ? *reinterpret_cast<const uint4 *>(x + k + 64 * h) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            we[i] = sw[i][b];
            xe[i] = sx[i][b];
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) multiply64(c, wv[h][0], wv[h][1], xv[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += scaled(c[i], we[i / 2], xe[i % 2]);
    }
    if (whole < b1) {
        const int64_t k = int64_t(whole) * kBlock;
        const float4 c = multiply_last(w[0] + k, w[1] + k, x + k, int(a.K - k) - 16 * t, token);
        sum[0] += scaled(c.x, sw[0][whole], sx[0][whole]);
        sum[1] += scaled(c.y, sw[0][whole], sx[1][whole]);
        sum[2] += scaled(c.z, sw[1][whole], sx[0][whole]);
        sum[3] += scaled(c.w, sw[1][whole], sx[1][whole]);
    }

    if (warps > 1) {
        part[warp][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        if (warp > 0) return;
        for (int i = 1; i < warps; ++i) {
            const float4 p = part[i][lane];
            sum[0] += p.x;
            sum[1] += p.y;
            sum[2] += p.z;
            sum[3] += p.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 2 * t + i % 2;
        const int64_t n = n0 + g + 8 * (i / 2);
        if (m >= a.M || n >= a.N) continue;
        if (a.bias != nullptr) sum[i] += Elem<T>::to_float(static_cast<const T *>(a.bias)[n]);
        T *c = static_cast<T *>(a.c) + m * a.c_stride + n;
        if (a.accumulate) sum[i] += Elem<T>::to_float(*c);
        *c = Elem<T>::from_float(sum[i]);
    }
}

template <class T> basp_status launch_matvec(MatvecArgs a, cudaStream_t stream) {
    // As many warps share K as fit the GPU at once, each with kVecBlocks blocks.
    const int64_t blocks = ceil_div(a.K, kBlock), groups = ceil_div(a.N, kVecRows), sms = sm_count();
    const dim3 grid{unsigned(groups)};
    // few rows, a long K (2048 x 8192: 4.7 us, 5.5 with eight warps)
    if (blocks >= 16 * kVecBlocks && groups <= sms)
        return launch(matvec_kernel<T, 16>, grid, dim3(16 * 32), 0, 1, stream, a);
    int warps = 1;
    while (warps < 8 && warps * 2 * kVecBlocks <= blocks && groups * warps * 2 <= sms * 24) warps *= 2;
    return launch(matvec_kernel<T, 8>, grid, dim3(unsigned(warps) * 32), 0, 1, stream, a);
}

}  // namespace basp_fp8
