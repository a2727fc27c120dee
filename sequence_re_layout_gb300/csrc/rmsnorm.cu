// rmsnorm.cu -- residual addition + root-mean-square norm with an 8-bit
// output, and its gradient (basp_rmsnorm, basp_rmsnorm_backward).
//
// Forward, for a row of n values:
//     h = x + residual,   rstd = (sum(h^2) / n + eps)^-1/2,   y = h * rstd * w
// and y in 8 bits with one scale for each 128 values.  Both reductions stay
// on the chip: a row's values are read once, held in registers from the sum
// of squares to the quantised store, and each 128-block belongs to one warp,
// whose lanes hold four values each, so the block's maximum is one warp
// reduction.  The bound is memory: 7 bytes a value for 16-bit types with a
// residual (two reads, h and the 8-bit value written).
//
// Backward, with g = dy * w and n = h * rstd (rstd does not depend on the row
// beyond h, d rstd / dh = -rstd^3 h / cols):
//     dx = rstd * (g - n * mean(g * n)) + dh,   dw = sum over rows of dy * n
// A CTA walks rows with a fixed stride and keeps its part of dw for its
// columns in registers; the CTAs' parts are summed by a second kernel in CTA
// order, so the result does not depend on timing.
#include <algorithm>

#include "fp8_common.cuh"

namespace basp_fp8 {

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 1;
    }
    return sms > 0 ? sms : 1;
}

namespace {

struct NormArgs {
    const void *x, *residual, *weight;
    void *h, *y;
    uint8_t *q, *scales;
    float *rstd;
    int64_t xs, rs, hs, ys, qs, ss;
    int64_t rows;
    int cols;
    bool vec16;
    float eps, inv_cols;
};

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

// y of one block, to memory in the forms asked for.
template <class T, class W, int HOW>
__device__ __forceinline__ void norm_store(const NormArgs &a, int64_t row, int b, int lane, int left,
                                           const float (&hv)[4], const float (&wv)[4], float rstd) {
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = hv[j] * rstd * wv[j];
    if (a.y != nullptr)
        store4<T, HOW>(static_cast<T *>(a.y) + row * a.ys + b * kBlock, lane, left, y);
    if (a.q != nullptr) {
        const uint32_t sb = row_scale(y);
        store4_e4m3<HOW>(a.q + row * a.qs + b * kBlock, lane, left, to_e4m3x4(y, inverse_scale(sb)));
        if (lane == 0) a.scales[row * a.ss + b] = uint8_t(sb);
    }
}

// NB > 0: warp w of a row's warps holds blocks w, w + warps, ... (NB of them)
// in registers.  NB = 0: rows too long for that; the row is walked twice.
// Rows that start anywhere (4099 x 5003 of 16 bits): 59 us with every access
// checked, 54 with whole blocks unchecked (43 instructions a value, not 55), 50
// with registers for five rows an SM instead of three; 21 us is memory's time.
template <class T, class W, int NB, bool VEC>
__global__ void __launch_bounds__(NB == 1 ? 1024 : 512, NB == 4 ? 3 : 1) norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float part[32];
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;            // whole warps; with several warps a row, blockDim.y is 1
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *r = a.residual ? static_cast<const T *>(a.residual) + row * a.rs : nullptr;
    const W *w = static_cast<const W *>(a.weight);
    T *h = a.h ? static_cast<T *>(a.h) + row * a.hs : nullptr;

    if constexpr (NB > 0) {
        float hv[NB][4], sq = 0.f;
        auto read = [&](auto how) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                load4<T, H>(x + c, lane, a.cols - c, hv[i]);
            }
            if (r != nullptr) {
                float rv[NB][4];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int c = (warp + i * warps) * kBlock;
                    load4<T, H>(r + c, lane, a.cols - c, rv[i]);
                }
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        hv[i][j] = Elem<T>::to_float(Elem<T>::from_float(hv[i][j] + rv[i][j]));
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                if (h != nullptr) store4<T, H>(h + c, lane, a.cols - c, hv[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sq += hv[i][j] * hv[i][j];
            }
        };
        auto write = [&](auto how, float rstd) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int b = warp + i * warps, c = b * kBlock;
                if (H != kWhole && c >= a.cols) break;
                float wv[4];
                load4<W, H>(w + c, lane, a.cols - c, wv);
                norm_store<T, W, H>(a, row, b, lane, a.cols - c, hv[i], wv, rstd);
            }
        };
        // a warp whose blocks all end inside the row needs no checks
        const bool whole = !VEC && (warp + (NB - 1) * warps + 1) * kBlock <= a.cols;
        if (whole) read(How<kWhole>());
        else read(How<VEC>());
        const float rstd = inverse_root(mean_of(row_sum(sq, part, warps), float(a.cols), a.inv_cols) + a.eps);
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
        if (whole) write(How<kWhole>(), rstd);
        else write(How<VEC>(), rstd);
    } else {
        auto load_h = [&](int c, float (&hv)[4]) {
            load4<T, VEC>(x + c, lane, a.cols - c, hv);
            if (r != nullptr) {
                float rv[4];
                load4<T, VEC>(r + c, lane, a.cols - c, rv);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    hv[j] = Elem<T>::to_float(Elem<T>::from_float(hv[j] + rv[j]));
            }
        };
        float sq = 0.f;
        for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += int64_t(warps) * kBlock) {
            float hv[4];
            load_h(int(c), hv);
            if (h != nullptr) store4<T, VEC>(h + c, lane, int(a.cols - c), hv);
#pragma unroll
            for (int j = 0; j < 4; ++j) sq += hv[j] * hv[j];
        }
        const float rstd = inverse_root(mean_of(row_sum(sq, part, warps), float(a.cols), a.inv_cols) + a.eps);
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
        for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += int64_t(warps) * kBlock) {
            float hv[4], wv[4];
            // h where it was written (it may be x or the residual itself), by
            // this very thread; else x + residual again
            if (h != nullptr) load4<T, VEC>(h + c, lane, int(a.cols - c), hv);
            else load_h(int(c), hv);
            load4<W, VEC>(w + c, lane, int(a.cols - c), wv);
            norm_store<T, W, VEC>(a, row, int(c / kBlock), lane, int(a.cols - c), hv, wv, rstd);
        }
    }
}

// The same for many rows that allow accesses of 16 bytes: the CTA walks rows
// with the grid's stride, and the loads of the next kAhead rows are on their
// way to shared memory while one is worked on, each thread copying what it
// will read itself.  A thread has NV vectors of 16 bytes, 8 or 4 values each;
// 16 or 32 neighbouring threads hold a 128-block.  The instructions count
// here: a value takes about 15, and 28 would be the bound instead of memory.
// 32768 x 2048 bf16 with a residual: 74 us, 6.3 TB/s, 0.93 of a copy's; the
// kernel above took 120.
constexpr int kAhead = 2;
constexpr int kWalkThreads = 512;

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

template <class T, class W, int NV>
__global__ void __launch_bounds__(kWalkThreads) norm_walk_kernel(const __grid_constant__ NormArgs a) {
    constexpr int ST = kAhead + 1, N = Pack<T>::N, G = kBlock / N;
    extern __shared__ __align__(16) uint8_t smem[];     // [stage][x, residual][vector][thread]
    __shared__ __align__(16) float part[2][16];
    const int threads = blockDim.x, warps = threads / 32;
    if (threadIdx.x < 32) part[threadIdx.x / 16][threadIdx.x % 16] = 0.f;
    uint4 *mine = reinterpret_cast<uint4 *>(smem) + threadIdx.x;
    grid_dependency();

    const T *x = static_cast<const T *>(a.x), *r = static_cast<const T *>(a.residual);
    int col[NV];
    bool have[NV];
    float wv[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * threads + int(threadIdx.x)) * N;
        have[i] = col[i] < a.cols;
#pragma unroll
        for (int j = 0; j < N; ++j)
            wv[i][j] = have[i] ? Elem<W>::to_float(static_cast<const W *>(a.weight)[col[i] + j]) : 0.f;
    }
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            const T *xr = x + row * a.xs, *rr = r + row * a.rs;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                copy16_async(mine + (stage * 2 * NV + i) * threads, have[i] ? xr + col[i] : x, have[i]);
                if (r != nullptr)
                    copy16_async(mine + (stage * 2 * NV + NV + i) * threads, have[i] ? rr + col[i] : r, have[i]);
            }
        }
        copy_commit();                    // an empty group past the end keeps the count
    };
    const int64_t step = gridDim.x;
    for (int i = 0; i < kAhead; ++i) fetch(blockIdx.x + i * step, i);
    __syncthreads();                      // part is zero

    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += step, turn ^= 1) {
        fetch(row + kAhead * step, stage >= 1 ? stage - 1 : ST - 1);
        copy_wait<kAhead>();
        float hv[NV][N], sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint4 raw = mine[(stage * 2 * NV + i) * threads];
            Pack<T>::unpack(raw, hv[i]);
            if (r != nullptr) {
                float f[N];
                Pack<T>::unpack(mine[(stage * 2 * NV + NV + i) * threads], f);
#pragma unroll
                for (int j = 0; j < N; ++j) hv[i][j] += f[j];
                raw = Pack<T>::pack(hv[i]);
                Pack<T>::unpack(raw, hv[i]);
            }
            if (a.h != nullptr && have[i])
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.h) + row * a.hs + col[i]) = raw;
#pragma unroll
            for (int j = 0; j < N; ++j) sq += hv[i][j] * hv[i][j];
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        // two buffers in turn: a warp can be one row ahead of another
        const float rstd = inverse_root(mean_of(walk_sum(sq, part[turn], warps), float(a.cols), a.inv_cols) + a.eps);
        if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
        // y, rounded after each factor as the definition has it: the row's number
        // of neighbours does not change how its values are rounded
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) hv[i][j] = hv[i][j] * rstd * wv[i][j];
        if (a.y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (have[i])
                    *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + row * a.ys + col[i]) = Pack<T>::pack(hv[i]);
        }
        if (a.q != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < N; ++j) top = fmaxf(top, fabsf(hv[i][j]));
                uint32_t m = block_max<G>(__float_as_uint(top));
                if (__any_sync(0xffffffffu, m >= kInfBits)) {    // an infinity: look at each value
                    uint32_t f = 0;
#pragma unroll
                    for (int j = 0; j < N; ++j) f = max(f, finite_bits(hv[i][j]));
                    m = block_max<G>(f);
                    infinite_to_nan(hv[i]);
                }
                const uint32_t sb = scale_byte(m);
                if (have[i]) {
                    store_e4m3<N>(a.q + row * a.qs + col[i], hv[i], inverse_scale(sb));
                    if (threadIdx.x % G == 0) a.scales[row * a.ss + col[i] / kBlock] = uint8_t(sb);
                }
            }
        }
    }
}

template <class T, class W, bool VEC>
basp_status launch_norm(const NormArgs &a, cudaStream_t stream) {
    const int blocks = int(ceil_div(a.cols, kBlock));
    // Few rows: a row is spread over as many warps as it has blocks.  Many:
    // four blocks a warp, which keeps 8 loads a thread in flight and the
    // cross-warp step small.
    const bool few = a.rows <= 2 * sm_count();
    if (a.vec16 && !few) {
        const int vectors = int(a.cols / Pack<T>::N);
        auto walk = [&](auto vectors_each) {
            constexpr int NV = decltype(vectors_each)::value;
            constexpr auto kernel = norm_walk_kernel<T, W, NV>;
            constexpr size_t per_thread = size_t(kAhead + 1) * 2 * NV * 16;
            if (!allow_shared_memory<kernel, per_thread * kWalkThreads>()) return BASP_ERR_CUDA;
            const int threads = int(ceil_div(vectors, NV * 32)) * 32;
            const size_t smem = per_thread * threads;
            const int64_t ctas = std::min(a.rows, resident_ctas(kernel, threads, smem));
            return launch(kernel, dim3(unsigned(ctas)), dim3(threads), smem, 1, stream, a);
        };
        if (vectors <= kWalkThreads) return walk(std::integral_constant<int, 1>());
        if (vectors <= 2 * kWalkThreads) return walk(std::integral_constant<int, 2>());
        if (vectors <= 4 * kWalkThreads) return walk(std::integral_constant<int, 4>());
    }
    if (blocks <= 4 && !few) {            // one warp a row, four rows a CTA
        return launch(norm_kernel<T, W, 4, VEC>, dim3(unsigned(ceil_div(a.rows, 4))), dim3(32, 4), 0, 1,
                      stream, a);
    }
    const dim3 grid(static_cast<unsigned>(a.rows));
    if (few && blocks <= 32)
        return launch(norm_kernel<T, W, 1, VEC>, grid, dim3(unsigned(blocks) * 32), 0, 1, stream, a);
    if (blocks <= 4 * 16)
        return launch(norm_kernel<T, W, 4, VEC>, grid, dim3(unsigned(ceil_div(blocks, 4)) * 32), 0, 1,
                      stream, a);
    return launch(norm_kernel<T, W, 0, VEC>, grid, dim3(512), 0, 1, stream, a);
}

struct NormBackArgs {
    const void *dy, *h, *weight, *dh;
    const float *rstd;
    void *dx;
    float *part;       // [gridDim.x][cols], or NULL
    int64_t dys, hs, dhs, dxs;
    int64_t rows;
    int cols;
    bool vec16;
    float inv_cols;
};

// NB blocks a warp, as above; the CTA walks rows blockIdx.x, + gridDim.x, ...
// Rows that start anywhere: 4099 x 5003 fp16 112 us, 32768 x 2047 bf16 187 (memory's
// time 24 and 79): checked accesses of single elements, and no row on its way
// while another is worked on.  NB = 0: 4096 x 16384 bf16 220 us (79).
template <class T, class W, int NB, bool VEC>
__global__ void __launch_bounds__(512) norm_back_kernel(const __grid_constant__ NormBackArgs a) {
    __shared__ float part[2][32];
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const W *w = static_cast<const W *>(a.weight);
    int turn = 0;
    if constexpr (NB > 0) {
        float wv[NB][4], dw[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int c = (warp + i * warps) * kBlock;
            load4<W, VEC>(w + c, lane, a.cols - c, wv[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) dw[i][j] = 0.f;
        }
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
            const T *h = static_cast<const T *>(a.h) + row * a.hs;
            const float rstd = a.rstd[row];
            float g[NB][4], n[NB][4];
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                load4<T, VEC>(dy + c, lane, a.cols - c, g[i]);
                load4<T, VEC>(h + c, lane, a.cols - c, n[i]);
            }
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[i][j] *= rstd;
                    dw[i][j] += g[i][j] * n[i][j];
                    g[i][j] *= wv[i][j];
                    dot += g[i][j] * n[i][j];
                }
            // two buffers in turn: a warp can be one row ahead of another
            const float mean = row_sum(dot, part[turn], warps) * a.inv_cols;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.dh != nullptr)
                    load4<T, VEC>(static_cast<const T *>(a.dh) + row * a.dhs + c, lane, a.cols - c, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rstd * (g[i][j] - n[i][j] * mean);
                store4<T, VEC>(static_cast<T *>(a.dx) + row * a.dxs + c, lane, a.cols - c, d);
            }
        }
        if (a.part != nullptr) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                store4<float, VEC>(a.part + int64_t(blockIdx.x) * a.cols + c, lane, a.cols - c, dw[i]);
            }
        }
    } else {
        // Rows too long for registers: two walks a row, the part of dw in
        // the CTA's own row of the workspace (each thread its own columns).
        float *dw = a.part ? a.part + int64_t(blockIdx.x) * a.cols : nullptr;
        const int64_t step = int64_t(warps) * kBlock;
        if (dw != nullptr)
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                store4<float, VEC>(dw + c, lane, int(a.cols - c), zero);
            }
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
            const T *h = static_cast<const T *>(a.h) + row * a.hs;
            const float rstd = a.rstd[row];
            float dot = 0.f;
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                float g[4], n[4], wv[4], s[4];
                const int left = int(a.cols - c);
                load4<T, VEC>(dy + c, lane, left, g);
                load4<T, VEC>(h + c, lane, left, n);
                load4<W, VEC>(w + c, lane, left, wv);
                if (dw != nullptr) load4<float, VEC>(dw + c, lane, left, s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] *= rstd;
                    if (dw != nullptr) s[j] += g[j] * n[j];
                    dot += g[j] * wv[j] * n[j];
                }
                if (dw != nullptr) store4<float, VEC>(dw + c, lane, left, s);
            }
            const float mean = row_sum(dot, part[turn], warps) * a.inv_cols;
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                float g[4], n[4], wv[4], d[4] = {0.f, 0.f, 0.f, 0.f};
                const int left = int(a.cols - c);
                load4<T, VEC>(dy + c, lane, left, g);
                load4<T, VEC>(h + c, lane, left, n);
                load4<W, VEC>(w + c, lane, left, wv);
                if (a.dh != nullptr) load4<T, VEC>(static_cast<const T *>(a.dh) + row * a.dhs + c, lane, left, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rstd * (g[j] * wv[j] - n[j] * rstd * mean);
                store4<T, VEC>(static_cast<T *>(a.dx) + row * a.dxs + c, lane, left, d);
            }
        }
    }
}

// The same for rows that allow accesses of 16 bytes, with the loads of the
// next kAhead rows on their way to shared memory.  32768 x 2048 bf16 with dh and
// dweight: 97 us, 5.5 TB/s, 0.82 of a copy's (163 without).
template <class T, class W, int NV>
__global__ void __launch_bounds__(kWalkThreads) norm_back_walk_kernel(const __grid_constant__ NormBackArgs a) {
    constexpr int ST = kAhead + 1, N = Pack<T>::N;
    extern __shared__ __align__(16) uint8_t smem[];     // [stage][dy, h, dh][vector][thread]
    __shared__ __align__(16) float part[2][16];
    const int threads = blockDim.x, warps = threads / 32;
    if (threadIdx.x < 32) part[threadIdx.x / 16][threadIdx.x % 16] = 0.f;
    uint4 *mine = reinterpret_cast<uint4 *>(smem) + threadIdx.x;
    grid_dependency();

    const T *dy = static_cast<const T *>(a.dy), *h = static_cast<const T *>(a.h);
    const T *dh = static_cast<const T *>(a.dh);
    int col[NV];
    bool have[NV];
    float wv[NV][N], dw[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * threads + int(threadIdx.x)) * N;
        have[i] = col[i] < a.cols;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            wv[i][j] = have[i] ? Elem<W>::to_float(static_cast<const W *>(a.weight)[col[i] + j]) : 0.f;
            dw[i][j] = 0.f;
        }
    }
    auto fetch = [&](int64_t row, int stage) {
        if (row < a.rows) {
            const T *d = dy + row * a.dys, *n = h + row * a.hs, *m = dh + row * a.dhs;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                uint4 *to = mine + (stage * 3 * NV + i) * threads;
                copy16_async(to, have[i] ? d + col[i] : dy, have[i]);
                copy16_async(to + NV * threads, have[i] ? n + col[i] : h, have[i]);
                if (dh != nullptr) copy16_async(to + 2 * NV * threads, have[i] ? m + col[i] : dh, have[i]);
            }
        }
        copy_commit();                    // an empty group past the end keeps the count
    };
    const int64_t step = gridDim.x;
    for (int i = 0; i < kAhead; ++i) fetch(blockIdx.x + i * step, i);
    __syncthreads();                      // part is zero

    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += step, turn ^= 1) {
        fetch(row + kAhead * step, stage >= 1 ? stage - 1 : ST - 1);
        const float rstd = a.rstd[row];
        copy_wait<kAhead>();
        const uint4 *at = mine + stage * 3 * NV * threads;
        float g[NV][N], n[NV][N], dot = 0.f;
        uint4 rest[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T>::unpack(at[i * threads], g[i]);
            Pack<T>::unpack(at[(NV + i) * threads], n[i]);
            rest[i] = dh != nullptr ? at[(2 * NV + i) * threads] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                n[i][j] *= rstd;
                dw[i][j] += g[i][j] * n[i][j];
                g[i][j] *= wv[i][j];
                dot += g[i][j] * n[i][j];
            }
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        const float mean = walk_sum(dot, part[turn], warps) * a.inv_cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float d[N];
            Pack<T>::unpack(rest[i], d);
#pragma unroll
            for (int j = 0; j < N; ++j) d[j] += rstd * (g[i][j] - n[i][j] * mean);
            if (have[i])
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dx) + row * a.dxs + col[i]) = Pack<T>::pack(d);
        }
    }
    if (a.part != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (have[i]) {
                float4 *out = reinterpret_cast<float4 *>(a.part + int64_t(blockIdx.x) * a.cols + col[i]);
#pragma unroll
                for (int j = 0; j < N / 4; ++j)
                    out[j] = make_float4(dw[i][4 * j], dw[i][4 * j + 1], dw[i][4 * j + 2], dw[i][4 * j + 3]);
            }
    }
}

// dweight[c] = sum over the parts' rows, in their order: 32 columns a CTA,
// 32 warps that each add every 32nd row, then one warp adds their sums.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *part, int parts, int cols, float *out) {
    __shared__ float s[32][33];
    grid_dependency();
    const int lane = threadIdx.x, warp = threadIdx.y;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float v = 0.f;
    if (c < cols)
        for (int p = warp; p < parts; p += 32) v += part[int64_t(p) * cols + c];
    s[warp][lane] = v;
    __syncthreads();
    v = warp_sum(s[lane][warp]);          // column `warp` of the CTA's 32
    const int64_t o = int64_t(blockIdx.x) * 32 + warp;
    if (lane == 0 && o < cols) out[o] = v;
}

// CTAs of the backward kernel: enough to fill the GPU four times over with
// rows of ordinary length, never more than there are rows.
constexpr int kBackCtasPerSm = 4;
constexpr int kBackMaxParts = 152 * kBackCtasPerSm;

int64_t back_parts(int64_t rows) { return std::min<int64_t>(rows, kBackMaxParts); }

template <class T, class W, bool VEC>
basp_status launch_norm_back(const NormBackArgs &a, cudaStream_t stream) {
    const int blocks = int(ceil_div(a.cols, kBlock));
    const dim3 grid(static_cast<unsigned>(back_parts(a.rows)));
    if (a.vec16) {
        const int vectors = int(a.cols / Pack<T>::N);
        auto walk = [&](auto vectors_each) {
            constexpr int NV = decltype(vectors_each)::value;
            constexpr auto kernel = norm_back_walk_kernel<T, W, NV>;
            constexpr size_t per_thread = size_t(kAhead + 1) * 3 * NV * 16;
            if (!allow_shared_memory<kernel, per_thread * kWalkThreads>()) return BASP_ERR_CUDA;
            const int threads = int(ceil_div(vectors, NV * 32)) * 32;
            return launch(kernel, grid, dim3(threads), per_thread * threads, 1, stream, a);
        };
        if (vectors <= kWalkThreads) return walk(std::integral_constant<int, 1>());
        if (vectors <= 2 * kWalkThreads) return walk(std::integral_constant<int, 2>());
    }
    if (blocks <= 32)
        return launch(norm_back_kernel<T, W, 2, VEC>, grid, dim3(unsigned(ceil_div(blocks, 2)) * 32), 0, 1,
                      stream, a);
    if (blocks <= 64)
        return launch(norm_back_kernel<T, W, 4, VEC>, grid, dim3(unsigned(ceil_div(blocks, 4)) * 32), 0, 1,
                      stream, a);
    return launch(norm_back_kernel<T, W, 0, VEC>, grid, dim3(512), 0, 1, stream, a);
}

// Calls f<T, W, VEC>() for the run-time types.
template <class F>
basp_status dispatch(basp_dtype t, basp_dtype w, bool vec, F &&f) {
    auto with = [&](auto te, auto we) {
        return vec ? f(te, we, std::true_type()) : f(te, we, std::false_type());
    };
    if (t == BASP_DTYPE_FP32) return with(float(), float());
    if (t == BASP_DTYPE_BF16)
        return w == BASP_DTYPE_FP32 ? with(__nv_bfloat16(), float()) : with(__nv_bfloat16(), __nv_bfloat16());
    return w == BASP_DTYPE_FP32 ? with(__half(), float()) : with(__half(), __half());
}

}  // namespace
}  // namespace basp_fp8

using namespace basp_fp8;

extern "C" basp_status basp_rmsnorm(basp_dtype dtype, int64_t rows, int64_t cols, const void *x,
                                    int64_t x_stride, const void *residual, int64_t residual_stride,
                                    const void *weight, basp_dtype weight_dtype, float eps, void *h,
                                    int64_t h_stride, void *y, int64_t y_stride,
                                    const basp_fp8_matrix *q, float *rstd, cudaStream_t stream) {
    NvtxRange range("basp_rmsnorm");
    basp_status st = BASP_OK;
    const int64_t esz = elem_size(dtype), wsz = elem_size(weight_dtype);
    if (esz == 0 || wsz == 0 || (weight_dtype != dtype && weight_dtype != BASP_DTYPE_FP32))
        return BASP_ERR_INVALID_ARG;
    if (!sides_ok(rows, cols, &st)) return st;
    if ((y == nullptr && q == nullptr) || !(eps >= 0.f)) return BASP_ERR_INVALID_ARG;
    Args args;
    args.matrix(x, rows, cols, x_stride, esz, false);
    args.matrix(residual, rows, cols, residual_stride, esz, false, false);
    args.matrix(weight, 1, cols, cols, wsz, false);
    args.matrix(h, rows, cols, h_stride, esz, true, false);
    args.matrix(y, rows, cols, y_stride, esz, true, false);
    args.matrix(rstd, 1, rows, rows, 4, true, false);
    if (q != nullptr) {
        if (q->block_rows != 1) return BASP_ERR_INVALID_ARG;
        args.fp8(q, rows, cols, true);
    }
    args.allow_same(h, x);
    args.allow_same(h, residual);
    st = args.status();
    if (st != BASP_OK || rows == 0 || cols == 0) return st;

    NormArgs a = {};
    a.x = x; a.residual = residual; a.weight = weight; a.h = h; a.y = y; a.rstd = rstd;
    a.xs = x_stride; a.rs = residual_stride; a.hs = h_stride; a.ys = y_stride;
    if (q != nullptr) {
        a.q = static_cast<uint8_t *>(q->data);
        a.scales = static_cast<uint8_t *>(q->scales);
        a.qs = q->pitch;
        a.ss = q->scale_pitch;
    }
    a.rows = rows; a.cols = int(cols); a.eps = eps; a.inv_cols = 1.f / float(cols);
    const bool vec = vec4_ok(x, x_stride, cols, esz) && vec4_ok(residual, residual_stride, cols, esz) &&
                     vec4_ok(weight, 0, cols, wsz) && vec4_ok(h, h_stride, cols, esz) &&
                     vec4_ok(y, y_stride, cols, esz);
    a.vec16 = vec16_ok(x, x_stride, cols, esz) && vec16_ok(residual, residual_stride, cols, esz) &&
              vec16_ok(h, h_stride, cols, esz) && vec16_ok(y, y_stride, cols, esz);
    return dispatch(dtype, weight_dtype, vec, [&](auto t, auto w, auto v) {
        return launch_norm<decltype(t), decltype(w), decltype(v)::value>(a, stream);
    });
}

extern "C" int64_t basp_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide) return 0;
    return back_parts(rows) * cols * int64_t(sizeof(float));
}

extern "C" basp_status basp_rmsnorm_backward(basp_dtype dtype, int64_t rows, int64_t cols, const void *dy,
                                             int64_t dy_stride, const void *h, int64_t h_stride,
                                             const float *rstd, const void *weight,
                                             basp_dtype weight_dtype, const void *dh, int64_t dh_stride,
                                             void *dx, int64_t dx_stride, float *dweight,
                                             void *workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
    NvtxRange range("basp_rmsnorm_backward");
    basp_status st = BASP_OK;
    const int64_t esz = elem_size(dtype), wsz = elem_size(weight_dtype);
    if (esz == 0 || wsz == 0 || (weight_dtype != dtype && weight_dtype != BASP_DTYPE_FP32))
        return BASP_ERR_INVALID_ARG;
    if (!sides_ok(rows, cols, &st)) return st;
    Args args;
    args.matrix(dy, rows, cols, dy_stride, esz, false);
    args.matrix(h, rows, cols, h_stride, esz, false);
    args.matrix(rstd, rows > 0 ? 1 : 0, rows, rows, 4, false, cols > 0);
    args.matrix(weight, 1, cols, cols, wsz, false);
    args.matrix(dh, rows, cols, dh_stride, esz, false, false);
    args.matrix(dx, rows, cols, dx_stride, esz, true);
    args.matrix(dweight, 1, cols, cols, 4, true, false);
    const int64_t need = dweight != nullptr ? basp_rmsnorm_backward_workspace(rows, cols) : 0;
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < size_t(need)) args.fail(BASP_ERR_WORKSPACE);
        else if (uintptr_t(workspace) % 16) args.fail(BASP_ERR_ALIGNMENT);
        else args.matrix(workspace, 1, need, need, 1, true);
    }
    args.allow_same(dx, dy);
    args.allow_same(dx, dh);
    st = args.status();
    if (st != BASP_OK || cols == 0) return st;
    if (rows == 0) {
        if (dweight != nullptr &&
            cudaMemsetAsync(dweight, 0, size_t(cols) * sizeof(float), stream) != cudaSuccess) {
            cudaGetLastError();
            return BASP_ERR_CUDA;
        }
        return BASP_OK;
    }

    NormBackArgs a = {};
    a.dy = dy; a.h = h; a.rstd = rstd; a.weight = weight; a.dh = dh; a.dx = dx;
    a.part = dweight != nullptr ? static_cast<float *>(workspace) : nullptr;
    a.dys = dy_stride; a.hs = h_stride; a.dhs = dh_stride; a.dxs = dx_stride;
    a.rows = rows; a.cols = int(cols); a.inv_cols = 1.f / float(cols);
    const bool vec = vec4_ok(dy, dy_stride, cols, esz) && vec4_ok(h, h_stride, cols, esz) &&
                     vec4_ok(weight, 0, cols, wsz) && vec4_ok(dh, dh_stride, cols, esz) &&
                     vec4_ok(dx, dx_stride, cols, esz);
    a.vec16 = vec16_ok(dy, dy_stride, cols, esz) && vec16_ok(h, h_stride, cols, esz) &&
              vec16_ok(dh, dh_stride, cols, esz) && vec16_ok(dx, dx_stride, cols, esz);
    st = dispatch(dtype, weight_dtype, vec, [&](auto t, auto w, auto v) {
        return launch_norm_back<decltype(t), decltype(w), decltype(v)::value>(a, stream);
    });
    if (st != BASP_OK || dweight == nullptr) return st;
    return launch(column_sum_kernel, dim3(unsigned(ceil_div(cols, 32))), dim3(32, 32), 0, 1, stream,
                  static_cast<const float *>(a.part), int(back_parts(rows)), int(cols), dweight);
}
