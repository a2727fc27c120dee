// layernorm.cu -- residual addition + layer norm with an 8-bit output, and its
// gradient (basp_layernorm, basp_layernorm_backward).
//
// Forward, for a row of n values:
//     h = x + residual,   mean = sum(h) / n,   var = sum((h - mean)^2) / n,
//     y = (h - mean) * (var + eps)^-1/2 * w + b
// The variance is taken about the mean, from values that stay in registers:
// sum(h^2) / n - mean^2 would lose every digit of a row whose mean is large.
//
// Backward, with g = dy * w and n = (h - mean) * rstd:
//     dx = rstd * (g - mean(g) - n * mean(g * n)) + dh,
//     dw = sum over rows of dy * n,   db = sum over rows of dy
// A CTA walks rows with a fixed stride and keeps its parts of dw and db for its
// columns in registers; a second kernel adds the CTAs' parts in their order.
//
// Both are bound by memory (7 and 8 bytes a value of 16-bit types with a
// residual), as the root-mean-square norm is, and are laid out like it.  32768 x 2048 bf16
// takes 79 us forward, with 8-bit y (0.89 of a copy's rate), and 102 backward (0.79).
#include <algorithm>

#include "norm_common.cuh"

namespace basp_fp8 {
namespace {

struct LayerArgs {
    const void *x, *residual, *weight, *bias;
    void *h, *y;
    uint8_t *q, *scales;
    float *mean, *rstd;
    int64_t xs, rs, hs, ys, qs, ss;
    int64_t rows;
    int cols;
    bool vec16;
    float eps, inv_cols;
};

// Whether lane `lane`'s value j of a 128-block (How of fp8_common.cuh) is one of
// its `left` columns.
template <int HOW> __device__ __forceinline__ bool inside(int lane, int j, int left) {
    return HOW == kWhole || (HOW == kVector ? 4 * lane + j : lane + 32 * j) < left;
}

template <class W, int HOW>
__device__ __forceinline__ void load4_or_zero(const W *p, int at, int lane, int left, float (&v)[4]) {
    if (p != nullptr) return load4<W, HOW>(p + at, lane, left, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 0.f;
}

// y of one block, to memory in the forms asked for.
template <class T, class W, int HOW>
__device__ __forceinline__ void layer_store(const LayerArgs &a, int64_t row, int b, int lane, int left,
                                            const float (&hv)[4], float mean, float rstd) {
    float y[4], w[4], c[4];
    load4<W, HOW>(static_cast<const W *>(a.weight) + b * kBlock, lane, left, w);
    load4_or_zero<W, HOW>(static_cast<const W *>(a.bias), b * kBlock, lane, left, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = inside<HOW>(lane, j, left) ? fmaf((hv[j] - mean) * rstd, w[j], c[j]) : 0.f;
    if (a.y != nullptr) store4<T, HOW>(static_cast<T *>(a.y) + row * a.ys + b * kBlock, lane, left, y);
    if (a.q != nullptr) {
        const uint32_t sb = row_scale(y);
        store4_e4m3<HOW>(a.q + row * a.qs + b * kBlock, lane, left, to_e4m3x4(y, inverse_scale(sb)));
        if (lane == 0) a.scales[row * a.ss + b] = uint8_t(sb);
    }
}

// NB > 0: warp w of a row's warps holds blocks w, w + warps, ... (NB of them) in
// registers.  NB = 0: rows too long for that, walked three times.
template <class T, class W, int NB, bool VEC>
__global__ void __launch_bounds__(NB == 1 ? 1024 : 512, NB == 4 ? 3 : 1) layer_kernel(const __grid_constant__ LayerArgs a) {
    __shared__ float part[2][32];
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int64_t row = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;            // whole warps; with several warps a row, blockDim.y is 1
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *r = a.residual ? static_cast<const T *>(a.residual) + row * a.rs : nullptr;
    T *h = a.h ? static_cast<T *>(a.h) + row * a.hs : nullptr;
    auto statistics = [&](float mean, float rstd) {
        if (threadIdx.x != 0) return;
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
    };

    if constexpr (NB > 0) {
        float hv[NB][4], sum = 0.f, dev = 0.f;
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
                for (int j = 0; j < 4; ++j) sum += hv[i][j];
            }
        };
        auto deviate = [&](auto how, float mean) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float d = hv[i][j] - mean;
                    if (inside<H>(lane, j, a.cols - (warp + i * warps) * kBlock)) dev += d * d;
                }
        };
        auto write = [&](auto how, float mean, float rstd) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int b = warp + i * warps, c = b * kBlock;
                if (H != kWhole && c >= a.cols) break;
                layer_store<T, W, H>(a, row, b, lane, a.cols - c, hv[i], mean, rstd);
            }
        };
        // a warp whose blocks all end inside the row needs no checks
        const bool whole = !VEC && (warp + (NB - 1) * warps + 1) * kBlock <= a.cols;
        if (whole) read(How<kWhole>());
        else read(How<VEC>());
        const float mean = mean_of(row_sum(sum, part[0], warps), float(a.cols), a.inv_cols);
        if (whole) deviate(How<kWhole>(), mean);
        else deviate(How<VEC>(), mean);
        const float rstd = inverse_root(mean_of(row_sum(dev, part[1], warps), float(a.cols), a.inv_cols) + a.eps);
        statistics(mean, rstd);
        if (whole) write(How<kWhole>(), mean, rstd);
        else write(How<VEC>(), mean, rstd);
    } else {
        auto load_h = [&](int64_t c, float (&hv)[4]) {
            // h where it was written (it may be x or the residual itself), by this
            // very thread
            load4<T, VEC>(x + c, lane, int(a.cols - c), hv);
            if (r != nullptr) {
                float rv[4];
                load4<T, VEC>(r + c, lane, int(a.cols - c), rv);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    hv[j] = Elem<T>::to_float(Elem<T>::from_float(hv[j] + rv[j]));
            }
        };
        const int64_t step = int64_t(warps) * kBlock;
        float sum = 0.f, dev = 0.f, hv[4];
        for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
            load_h(c, hv);
            if (h != nullptr) store4<T, VEC>(h + c, lane, int(a.cols - c), hv);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += hv[j];
        }
        const float mean = mean_of(row_sum(sum, part[0], warps), float(a.cols), a.inv_cols);
        auto again = [&](int64_t c) {
            if (h != nullptr) load4<T, VEC>(h + c, lane, int(a.cols - c), hv);
            else load_h(c, hv);
        };
        for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
            again(c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = hv[j] - mean;
                if (inside<VEC>(lane, j, int(a.cols - c))) dev += d * d;
            }
        }
        const float rstd = inverse_root(mean_of(row_sum(dev, part[1], warps), float(a.cols), a.inv_cols) + a.eps);
        statistics(mean, rstd);
        for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
            again(c);
            layer_store<T, W, VEC>(a, row, int(c / kBlock), lane, int(a.cols - c), hv, mean, rstd);
        }
    }
}

// The same for many rows that allow accesses of 16 bytes: the CTA walks rows
// with the grid's stride, and the loads of the next kAhead rows are on their
// way to shared memory while one is worked on, each thread copying what it
// will read itself.  A warp takes the mean of its own values and their squares
// about that; one barrier a row, after which
//     sum (h - mean)^2 = sum over warps of (M2 + count * (mean_w - mean)^2).
template <class T, class W, int NV>
__global__ void __launch_bounds__(kWalkThreads) layer_walk_kernel(const __grid_constant__ LayerArgs a) {
    constexpr int ST = kAhead + 1, N = Pack<T>::N, G = kBlock / N;
    extern __shared__ __align__(16) uint8_t smem[];     // [stage][x, residual][vector][thread]
    __shared__ float4 part[2][16];                      // sum, M2, mean and count of a warp; zero past the last
    const int threads = blockDim.x, warps = threads / 32, lane = threadIdx.x % 32;
    if (threadIdx.x < 32) part[threadIdx.x / 16][threadIdx.x % 16] = make_float4(0.f, 0.f, 0.f, 0.f);
    uint4 *mine = reinterpret_cast<uint4 *>(smem) + threadIdx.x;
    grid_dependency();

    const T *x = static_cast<const T *>(a.x), *r = static_cast<const T *>(a.residual);
    int col[NV], count = 0;
    bool have[NV];
    float wv[NV][N], bv[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * threads + int(threadIdx.x)) * N;
        have[i] = col[i] < a.cols;
        count += __popc(__ballot_sync(0xffffffffu, have[i])) * N;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            wv[i][j] = have[i] ? Elem<W>::to_float(static_cast<const W *>(a.weight)[col[i] + j]) : 0.f;
            bv[i][j] = have[i] && a.bias != nullptr ? Elem<W>::to_float(static_cast<const W *>(a.bias)[col[i] + j]) : 0.f;
        }
    }
    const float inv_count = 1.f / float(count);         // a warp has one vector at least
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
        float hv[NV][N], sum = 0.f;
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
            for (int j = 0; j < N; ++j) sum += hv[i][j];
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        sum = warp_sum(sum);
        const float own = sum * inv_count;
        float dev = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float d = hv[i][j] - own;
                if (have[i]) dev += d * d;
            }
        dev = warp_sum(dev);
        float mean = own;
        if (warps > 1) {
            // two buffers in turn: a warp can be one row ahead of another
            if (lane == 0) part[turn][threadIdx.x / 32] = make_float4(sum, dev, own, float(count));
            __syncthreads();
            const float4 p = part[turn][lane % 16];
            sum = p.x;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mean = mean_of(sum, float(a.cols), a.inv_cols);
            dev = p.w > 0.f ? p.y + p.w * (p.z - mean) * (p.z - mean) : 0.f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) dev += __shfl_xor_sync(0xffffffffu, dev, o);
        } else {
            mean = mean_of(sum, float(a.cols), a.inv_cols);
        }
        const float rstd = inverse_root(mean_of(dev, float(a.cols), a.inv_cols) + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean != nullptr) a.mean[row] = mean;
            if (a.rstd != nullptr) a.rstd[row] = rstd;
        }
        // y, rounded as in the kernel above
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) hv[i][j] = fmaf((hv[i][j] - mean) * rstd, wv[i][j], bv[i][j]);   // past the end: 0
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
basp_status launch_layer(const LayerArgs &a, cudaStream_t stream) {
    const int blocks = int(ceil_div(a.cols, kBlock));
    // Few rows: a row is spread over as many warps as it has blocks.
    const bool few = a.rows <= 2 * sm_count();
    if (a.vec16 && !few) {
        const int vectors = int(a.cols / Pack<T>::N);
        auto walk = [&](auto vectors_each) {
            constexpr int NV = decltype(vectors_each)::value;
            constexpr auto kernel = layer_walk_kernel<T, W, NV>;
            constexpr size_t per_thread = size_t(kAhead + 1) * 2 * NV * 16;
            if (!allow_shared_memory<kernel, per_thread * kWalkThreads>()) return BASP_ERR_CUDA;
            const int threads = int(ceil_div(vectors, NV * 32)) * 32;
            const size_t smem = per_thread * threads;
            const int64_t ctas = std::min(a.rows, resident_ctas(kernel, threads, smem));
            return launch(kernel, dim3(unsigned(ctas)), dim3(threads), smem, 1, stream, a);
        };
        // What a row costs beside its values (sums over lanes and warps, a root) is the
        // smaller part the more values a thread has: 32768 x 2048 bf16 takes 97 us with one
        // vector a thread, 87 with two, 79 with four.
        if (vectors <= 32) return walk(std::integral_constant<int, 1>());
        if (vectors <= 64) return walk(std::integral_constant<int, 2>());
        if (vectors <= 4 * kWalkThreads) return walk(std::integral_constant<int, 4>());
    }
    if (blocks <= 4 && !few)              // one warp a row, four rows a CTA
        return launch(layer_kernel<T, W, 4, VEC>, dim3(unsigned(ceil_div(a.rows, 4))), dim3(32, 4), 0, 1, stream, a);
    const dim3 grid(static_cast<unsigned>(a.rows));
    if (few && blocks <= 32)
        return launch(layer_kernel<T, W, 1, VEC>, grid, dim3(unsigned(blocks) * 32), 0, 1, stream, a);
    if (blocks <= 4 * 16)
        return launch(layer_kernel<T, W, 4, VEC>, grid, dim3(unsigned(ceil_div(blocks, 4)) * 32), 0, 1, stream, a);
    return launch(layer_kernel<T, W, 0, VEC>, grid, dim3(512), 0, 1, stream, a);
}

// ---- backward -------------------------------------------------------------------

struct LayerBackArgs {
    const void *dy, *h, *weight, *dh;
    const float *mean, *rstd;
    void *dx;
    float *part;       // [gridDim.x][dw of cols, db of cols], or NULL
    int64_t dys, hs, dhs, dxs;
    int64_t rows;
    int cols;
    bool vec16;
    float inv_cols;
};

// Two sums over all warps of the CTA's row, the same in every thread.  `part` has
// room for 32 and is zero past the CTA's warps.
__device__ __forceinline__ float2 row_sum2(float a, float b, float2 *part, int warps) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (warps == 1) return make_float2(a, b);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
    for (int i = 0; i < warps; i += 2) {
        const float4 p = *reinterpret_cast<const float4 *>(part + i);
        a += p.x + p.z;
        b += p.y + p.w;
    }
    return make_float2(a, b);
}

// NB blocks a warp, as above; the CTA walks rows blockIdx.x, + gridDim.x, ...
template <class T, class W, int NB, bool VEC, int THREADS = 512>
__global__ void __launch_bounds__(THREADS) layer_back_kernel(const __grid_constant__ LayerBackArgs a) {
    __shared__ __align__(16) float2 part[2][32];
    for (int i = threadIdx.x; i < 64; i += blockDim.x) part[i / 32][i % 32] = make_float2(0.f, 0.f);
    __syncthreads();
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const W *w = static_cast<const W *>(a.weight);
    int turn = 0;
    if constexpr (NB > 0) {
        float wv[NB][4], dw[NB][4], db[NB][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int c = (warp + i * warps) * kBlock;
            load4<W, VEC>(w + c, lane, a.cols - c, wv[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0.f;
        }
        // a warp whose blocks all end inside the row needs no checks; the barrier of the row's
        // sums is for all warps, and so outside of what they do differently
        const bool whole = !VEC && (warp + (NB - 1) * warps + 1) * kBlock <= a.cols;
        float g[NB][4], n[NB][4], dot, all;
        auto read = [&](auto how, const T *dy, const T *h, float mean, float rstd) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                load4<T, H>(dy + c, lane, a.cols - c, g[i]);
                load4<T, H>(h + c, lane, a.cols - c, n[i]);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = inside<H>(lane, j, a.cols - (warp + i * warps) * kBlock);
                    n[i][j] = in ? (n[i][j] - mean) * rstd : 0.f;
                    dw[i][j] += g[i][j] * n[i][j];
                    db[i][j] += g[i][j];
                    g[i][j] *= wv[i][j];
                    all += g[i][j];
                    dot += g[i][j] * n[i][j];
                }
        };
        auto write = [&](auto how, const T *dh, T *dx, float mg, float mn, float rstd) {
            constexpr int H = decltype(how)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.dh != nullptr) load4<T, H>(dh + c, lane, a.cols - c, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rstd * (g[i][j] - mg - n[i][j] * mn);
                store4<T, H>(dx + c, lane, a.cols - c, d);
            }
        };
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            const T *dy = static_cast<const T *>(a.dy) + row * a.dys, *h = static_cast<const T *>(a.h) + row * a.hs;
            const T *dh = static_cast<const T *>(a.dh) + row * a.dhs;
            T *dx = static_cast<T *>(a.dx) + row * a.dxs;
            const float mean = a.mean[row], rstd = a.rstd[row];
            dot = all = 0.f;
            if (whole) read(How<kWhole>(), dy, h, mean, rstd);
            else read(How<VEC>(), dy, h, mean, rstd);
            // two buffers in turn: a warp can be one row ahead of another
            const float2 s = row_sum2(all, dot, part[turn], warps);
            const float mg = s.x * a.inv_cols, mn = s.y * a.inv_cols;
            if (whole) write(How<kWhole>(), dh, dx, mg, mn, rstd);
            else write(How<VEC>(), dh, dx, mg, mn, rstd);
        }
        if (a.part != nullptr) {
            float *to = a.part + int64_t(blockIdx.x) * 2 * a.cols;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (warp + i * warps) * kBlock;
                store4<float, VEC>(to + c, lane, a.cols - c, dw[i]);
                store4<float, VEC>(to + a.cols + c, lane, a.cols - c, db[i]);
            }
        }
    } else {
        // Rows too long for registers: two walks a row, the parts of dw and db in
        // the CTA's own row of the workspace (each thread its own columns).
        float *dw = a.part ? a.part + int64_t(blockIdx.x) * 2 * a.cols : nullptr, *db = dw + a.cols;
        const int64_t step = int64_t(warps) * kBlock;
        if (dw != nullptr)
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                store4<float, VEC>(dw + c, lane, int(a.cols - c), zero);
                store4<float, VEC>(db + c, lane, int(a.cols - c), zero);
            }
        for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
            const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
            const T *h = static_cast<const T *>(a.h) + row * a.hs;
            const float mean = a.mean[row], rstd = a.rstd[row];
            float dot = 0.f, all = 0.f;
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                float g[4], n[4], wv[4], s[4], t[4];
                const int left = int(a.cols - c);
                load4<T, VEC>(dy + c, lane, left, g);
                load4<T, VEC>(h + c, lane, left, n);
                load4<W, VEC>(w + c, lane, left, wv);
                if (dw != nullptr) {
                    load4<float, VEC>(dw + c, lane, left, s);
                    load4<float, VEC>(db + c, lane, left, t);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    n[j] = inside<VEC>(lane, j, left) ? (n[j] - mean) * rstd : 0.f;
                    if (dw != nullptr) {
                        s[j] += g[j] * n[j];
                        t[j] += g[j];
                    }
                    all += g[j] * wv[j];
                    dot += g[j] * wv[j] * n[j];
                }
                if (dw != nullptr) {
                    store4<float, VEC>(dw + c, lane, left, s);
                    store4<float, VEC>(db + c, lane, left, t);
                }
            }
            const float2 s = row_sum2(all, dot, part[turn], warps);
            const float mg = s.x * a.inv_cols, mn = s.y * a.inv_cols;
            for (int64_t c = int64_t(warp) * kBlock; c < a.cols; c += step) {
                float g[4], n[4], wv[4], d[4] = {0.f, 0.f, 0.f, 0.f};
                const int left = int(a.cols - c);
                load4<T, VEC>(dy + c, lane, left, g);
                load4<T, VEC>(h + c, lane, left, n);
                load4<W, VEC>(w + c, lane, left, wv);
                if (a.dh != nullptr) load4<T, VEC>(static_cast<const T *>(a.dh) + row * a.dhs + c, lane, left, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] += rstd * (g[j] * wv[j] - mg - (n[j] - mean) * rstd * mn);
                store4<T, VEC>(static_cast<T *>(a.dx) + row * a.dxs + c, lane, left, d);
            }
        }
    }
}

// The same for rows that allow accesses of 16 bytes, with the loads of the
// next AHEAD rows on their way to shared memory.
template <class T, class W, int NV, int AHEAD>
__global__ void __launch_bounds__(kWalkThreads) layer_back_walk_kernel(const __grid_constant__ LayerBackArgs a) {
    constexpr int ST = AHEAD + 1, N = Pack<T>::N;
    extern __shared__ __align__(16) uint8_t smem[];     // [stage][dy, h, dh][vector][thread]
    __shared__ __align__(16) float2 part[2][32];
    const int threads = blockDim.x, warps = threads / 32;
    if (threadIdx.x < 32) part[0][threadIdx.x] = part[1][threadIdx.x] = make_float2(0.f, 0.f);
    uint4 *mine = reinterpret_cast<uint4 *>(smem) + threadIdx.x;
    grid_dependency();

    const T *dy = static_cast<const T *>(a.dy), *h = static_cast<const T *>(a.h);
    const T *dh = static_cast<const T *>(a.dh);
    int col[NV];
    bool have[NV];
    float wv[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * threads + int(threadIdx.x)) * N;
        have[i] = col[i] < a.cols;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            wv[i][j] = have[i] ? Elem<W>::to_float(static_cast<const W *>(a.weight)[col[i] + j]) : 0.f;
            dw[i][j] = db[i][j] = 0.f;
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
    for (int i = 0; i < AHEAD; ++i) fetch(blockIdx.x + i * step, i);
    __syncthreads();                      // part is zero

    int stage = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += step, turn ^= 1) {
        fetch(row + AHEAD * step, stage >= 1 ? stage - 1 : ST - 1);
        const float mean = a.mean[row], rstd = a.rstd[row];
        copy_wait<AHEAD>();
        const uint4 *at = mine + stage * 3 * NV * threads;
        float g[NV][N], n[NV][N], dot = 0.f, all = 0.f;
        uint4 rest[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T>::unpack(at[i * threads], g[i]);
            Pack<T>::unpack(at[(NV + i) * threads], n[i]);
            rest[i] = dh != nullptr ? at[(2 * NV + i) * threads] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                n[i][j] = (n[i][j] - mean) * rstd;       // past the row's end it meets g = 0
                dw[i][j] += g[i][j] * n[i][j];
                db[i][j] += g[i][j];
                g[i][j] *= wv[i][j];
                all += g[i][j];
                dot += have[i] ? g[i][j] * n[i][j] : 0.f;
            }
        }
        stage = stage + 1 < ST ? stage + 1 : 0;
        const float2 s = row_sum2(all, dot, part[turn], warps);
        const float mg = s.x * a.inv_cols, mn = s.y * a.inv_cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float d[N];
            Pack<T>::unpack(rest[i], d);
#pragma unroll
            for (int j = 0; j < N; ++j) d[j] += rstd * (g[i][j] - mg - n[i][j] * mn);
            if (have[i])
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dx) + row * a.dxs + col[i]) = Pack<T>::pack(d);
        }
    }
    if (a.part != nullptr) {
        float *to = a.part + int64_t(blockIdx.x) * 2 * a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (have[i]) {
                float4 *ow = reinterpret_cast<float4 *>(to + col[i]), *ob = reinterpret_cast<float4 *>(to + a.cols + col[i]);
#pragma unroll
                for (int j = 0; j < N / 4; ++j) {
                    ow[j] = make_float4(dw[i][4 * j], dw[i][4 * j + 1], dw[i][4 * j + 2], dw[i][4 * j + 3]);
                    ob[j] = make_float4(db[i][4 * j], db[i][4 * j + 1], db[i][4 * j + 2], db[i][4 * j + 3]);
                }
            }
    }
}

// The parts' rows added in their order, dw's columns and then db's: 32 columns a
// CTA, 32 warps that each add every 32nd row, then one warp adds their sums.
__global__ void __launch_bounds__(1024) layer_column_sum_kernel(const float *part, int parts, int cols, float *dw, float *db) {
    __shared__ float s[32][33];
    grid_dependency();
    const int lane = threadIdx.x, warp = threadIdx.y;
    const int64_t width = 2 * int64_t(cols), c = int64_t(blockIdx.x) * 32 + lane;
    float v = 0.f;
    if (c < width)
        for (int p = warp; p < parts; p += 32) v += part[p * width + c];
    s[warp][lane] = v;
    __syncthreads();
    v = warp_sum(s[lane][warp]);          // column `warp` of the CTA's 32
    const int64_t o = int64_t(blockIdx.x) * 32 + warp;
    if (lane == 0 && o < cols && dw != nullptr) dw[o] = v;
    if (lane == 0 && o >= cols && o < width && db != nullptr) db[o - cols] = v;
}

// CTAs of the backward kernel, and parts of dw and db: never more than fit at once, than
// there are rows, or than the workspace has room for.  Narrow rows have small CTAs, which
// are more: 60000 x 512 bf16 took 104 us with four an SM.
int64_t back_parts(int64_t rows, int64_t cols) {
    return std::min<int64_t>(rows, kSms * std::min<int64_t>(16, std::max<int64_t>(4, 8192 / cols)));
}

template <class T, class W, bool VEC>
basp_status launch_layer_back(const LayerBackArgs &a, int64_t *parts, cudaStream_t stream) {
    const int blocks = int(ceil_div(a.cols, kBlock));
    auto go = [&](auto kernel, int threads, size_t smem) {
        *parts = std::min(back_parts(a.rows, a.cols), resident_ctas(kernel, threads, smem));
        return launch(kernel, dim3(unsigned(*parts)), dim3(threads), smem, 1, stream, a);
    };
    if (a.vec16) {
        const int vectors = int(a.cols / Pack<T>::N);
        auto walk = [&](auto vectors_each) {
            constexpr int NV = decltype(vectors_each)::value, AHEAD = NV == 4 ? 1 : kAhead;
            constexpr auto kernel = layer_back_walk_kernel<T, W, NV, AHEAD>;
            constexpr size_t per_thread = size_t(AHEAD + 1) * 3 * NV * 16;
            if (!allow_shared_memory<kernel, per_thread * kWalkThreads>()) return BASP_ERR_CUDA;
            const int threads = int(ceil_div(vectors, NV * 32)) * 32;
            return go(kernel, threads, per_thread * threads);
        };
        // 16 values a thread: 8192 x 4096 fp32 takes 115 us with two vectors, 85 with four;
        // 32768 x 2048 bf16 102 with two, 232 with four, which leave no registers
        if (vectors <= 32) return walk(std::integral_constant<int, 1>());
        if (vectors <= (Pack<T>::N == 8 ? 2 * kWalkThreads : 64)) return walk(std::integral_constant<int, 2>());
        if (vectors <= 4 * kWalkThreads) return walk(std::integral_constant<int, 4>());
    }
    const int threads = int(ceil_div(blocks, 2)) * 32;
    if (threads <= 512) return go(layer_back_kernel<T, W, 2, VEC>, threads, 0);
    if (threads <= 768) return go(layer_back_kernel<T, W, 2, VEC, 768>, threads, 0);
    if (threads <= 1024) return go(layer_back_kernel<T, W, 2, VEC, 1024>, threads, 0);
    return go(layer_back_kernel<T, W, 0, VEC>, 512, 0);
}

}  // namespace
}  // namespace basp_fp8

using namespace basp_fp8;

extern "C" basp_status basp_layernorm(basp_dtype dtype, int64_t rows, int64_t cols, const void *x,
                                      int64_t x_stride, const void *residual, int64_t residual_stride,
                                      const void *weight, const void *bias, basp_dtype weight_dtype, float eps,
                                      void *h, int64_t h_stride, void *y, int64_t y_stride,
                                      const basp_fp8_matrix *q, float *mean, float *rstd, cudaStream_t stream) {
    NvtxRange range("basp_layernorm");
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
    args.matrix(bias, 1, cols, cols, wsz, false, false);
    args.matrix(h, rows, cols, h_stride, esz, true, false);
    args.matrix(y, rows, cols, y_stride, esz, true, false);
    args.matrix(mean, 1, rows, rows, 4, true, false);
    args.matrix(rstd, 1, rows, rows, 4, true, false);
    if (q != nullptr) {
        if (q->block_rows != 1) return BASP_ERR_INVALID_ARG;
        args.fp8(q, rows, cols, true);
    }
    args.allow_same(h, x);
    args.allow_same(h, residual);
    st = args.status();
    if (st != BASP_OK || rows == 0 || cols == 0) return st;

    LayerArgs a = {};
    a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.h = h; a.y = y; a.mean = mean; a.rstd = rstd;
    a.xs = x_stride; a.rs = residual_stride; a.hs = h_stride; a.ys = y_stride;
    if (q != nullptr) {
        a.q = static_cast<uint8_t *>(q->data);
        a.scales = static_cast<uint8_t *>(q->scales);
        a.qs = q->pitch;
        a.ss = q->scale_pitch;
    }
    a.rows = rows; a.cols = int(cols); a.eps = eps; a.inv_cols = 1.f / float(cols);
    const bool vec = vec4_ok(x, x_stride, cols, esz) && vec4_ok(residual, residual_stride, cols, esz) &&
                     vec4_ok(weight, 0, cols, wsz) && vec4_ok(bias, 0, cols, wsz) &&
                     vec4_ok(h, h_stride, cols, esz) && vec4_ok(y, y_stride, cols, esz);
    a.vec16 = vec16_ok(x, x_stride, cols, esz) && vec16_ok(residual, residual_stride, cols, esz) &&
              vec16_ok(h, h_stride, cols, esz) && vec16_ok(y, y_stride, cols, esz);
    return dispatch(dtype, weight_dtype, vec, [&](auto t, auto w, auto v) {
        return launch_layer<decltype(t), decltype(w), decltype(v)::value>(a, stream);
    });
}

extern "C" int64_t basp_layernorm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kMaxSide || cols > kMaxSide) return 0;
    return back_parts(rows, cols) * 2 * cols * int64_t(sizeof(float));
}

extern "C" basp_status basp_layernorm_backward(basp_dtype dtype, int64_t rows, int64_t cols, const void *dy,
                                               int64_t dy_stride, const void *h, int64_t h_stride,
                                               const float *mean, const float *rstd, const void *weight,
                                               basp_dtype weight_dtype, const void *dh, int64_t dh_stride,
                                               void *dx, int64_t dx_stride, float *dweight, float *dbias,
                                               void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange range("basp_layernorm_backward");
    basp_status st = BASP_OK;
    const int64_t esz = elem_size(dtype), wsz = elem_size(weight_dtype);
    if (esz == 0 || wsz == 0 || (weight_dtype != dtype && weight_dtype != BASP_DTYPE_FP32))
        return BASP_ERR_INVALID_ARG;
    if (!sides_ok(rows, cols, &st)) return st;
    const bool sums = dweight != nullptr || dbias != nullptr;
    Args args;
    args.matrix(dy, rows, cols, dy_stride, esz, false);
    args.matrix(h, rows, cols, h_stride, esz, false);
    args.matrix(mean, rows > 0 ? 1 : 0, rows, rows, 4, false, cols > 0);
    args.matrix(rstd, rows > 0 ? 1 : 0, rows, rows, 4, false, cols > 0);
    args.matrix(weight, 1, cols, cols, wsz, false);
    args.matrix(dh, rows, cols, dh_stride, esz, false, false);
    args.matrix(dx, rows, cols, dx_stride, esz, true);
    args.matrix(dweight, 1, cols, cols, 4, true, false);
    args.matrix(dbias, 1, cols, cols, 4, true, false);
    const int64_t need = sums ? basp_layernorm_backward_workspace(rows, cols) : 0;
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
        for (float *p : {dweight, dbias})
            if (p != nullptr && cudaMemsetAsync(p, 0, size_t(cols) * sizeof(float), stream) != cudaSuccess) {
                cudaGetLastError();
                return BASP_ERR_CUDA;
            }
        return BASP_OK;
    }

    LayerBackArgs a = {};
    a.dy = dy; a.h = h; a.mean = mean; a.rstd = rstd; a.weight = weight; a.dh = dh; a.dx = dx;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    a.dys = dy_stride; a.hs = h_stride; a.dhs = dh_stride; a.dxs = dx_stride;
    a.rows = rows; a.cols = int(cols); a.inv_cols = 1.f / float(cols);
    const bool vec = vec4_ok(dy, dy_stride, cols, esz) && vec4_ok(h, h_stride, cols, esz) &&
                     vec4_ok(weight, 0, cols, wsz) && vec4_ok(dh, dh_stride, cols, esz) &&
                     vec4_ok(dx, dx_stride, cols, esz);
    a.vec16 = vec16_ok(dy, dy_stride, cols, esz) && vec16_ok(h, h_stride, cols, esz) &&
              vec16_ok(dh, dh_stride, cols, esz) && vec16_ok(dx, dx_stride, cols, esz);
    int64_t parts = 0;
    st = dispatch(dtype, weight_dtype, vec, [&](auto t, auto w, auto v) {
        return launch_layer_back<decltype(t), decltype(w), decltype(v)::value>(a, &parts, stream);
    });
    if (st != BASP_OK || !sums) return st;
    return launch(layer_column_sum_kernel, dim3(unsigned(ceil_div(2 * cols, 32))), dim3(32, 32), 0, 1, stream,
                  static_cast<const float *>(a.part), int(parts), int(cols), dweight, dbias);
}
