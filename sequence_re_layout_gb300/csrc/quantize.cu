// quantize.cu -- 16- and 32-bit matrices to e4m3 with a power-of-two scale for
// each 1 x 128 or 128 x 128 block, and the same for the transpose
// (basp_quantize_fp8).
//
// Each value is read once whatever is asked for: the bound is memory (3 bytes
// a value for a 16-bit matrix, 4 with the transpose), if the instructions stay
// few.  Rows alone need no tile: a warp owns 128-blocks, four values a lane.
// The transpose and 128 x 128 scales work on 128 x 128 tiles: a lane holds a
// few columns of a few rows, so that row maxima join lanes of one warp, column
// maxima join warps in shared memory, and four rows of a column are four
// consecutive bytes of the transpose, which go through shared memory to leave
// as 128-byte rows.
#include <algorithm>

#include "fp8_common.cuh"

namespace basp_fp8 {
namespace {

struct QuantArgs {
    const void *x;
    uint8_t *q, *scales, *qt, *scales_t;
    int64_t xs, qs, ss, qts, sts;
    int64_t rows;
    int cols;
};

// ---- rows alone -----------------------------------------------------------

constexpr int kRowWarps = 8;       // warps a CTA
constexpr int kRowBlocks = 4;      // 128-blocks a warp: loads in flight

// Warp units are groups of kRowBlocks neighbouring blocks of one row.  32768 x 2048
// bf16: 63 us, 30 memory's time: a warp ends after four blocks, and nothing is on
// its way while they are rounded.
template <class T, bool VEC>
__global__ void __launch_bounds__(kRowWarps * 32)
quantize_rows_kernel(const __grid_constant__ QuantArgs a, int groups) {
    grid_dependency();
    const int lane = threadIdx.x % 32;
    const int64_t unit = int64_t(blockIdx.x) * kRowWarps + threadIdx.x / 32;
    const int64_t row = unit / groups;
    const int b0 = int(unit % groups) * kRowBlocks;
    if (row >= a.rows) return;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    float v[kRowBlocks][4];
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
        const int64_t c = int64_t(b0 + i) * kBlock;
        if (c < a.cols) load4<T, VEC>(x + c, lane, int(a.cols - c), v[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowBlocks; ++i) {
        const int64_t c = int64_t(b0 + i) * kBlock;
        if (c >= a.cols) break;
        const uint32_t sb = row_scale(v[i]);
        store4_e4m3<VEC>(a.q + row * a.qs + c, lane, int(a.cols - c), to_e4m3x4(v[i], inverse_scale(sb)));
        if (lane == 0) a.scales[row * a.ss + b0 + i] = uint8_t(sb);
    }
}

// ---- tiles ----------------------------------------------------------------

constexpr int kTileWarps = 8;
constexpr int kTileThreads = kTileWarps * 32;
constexpr int kTileRows = kBlock / kTileWarps;      // rows a warp
constexpr int kTileAhead = 1;                       // tiles whose loads are on their way

// Where 4-byte piece p (of 32) of transposed row n sits in its 128 bytes of
// shared memory: neighbouring lanes, whose n differ by 1, 4 or 8, store to the
// eight 16-byte groups in turn, and a group's four pieces stay together for
// the loads.
__device__ __forceinline__ int piece(int n, int p) { return p ^ ((((n >> 3) ^ n) & 7) << 2); }

// The transpose's tile from shared memory: 16 bytes a thread, eight threads a
// row.
__device__ __forceinline__ void store_transposed(const QuantArgs &a, const uint8_t *t, int64_t m0, int64_t n0,
                                                 int left_m, int left_n) {
#pragma unroll
    for (int k = 0; k < kBlock * kBlock / (16 * kTileThreads); ++k) {
        const int n = k * (kTileThreads / 8) + int(threadIdx.x) / 8, w = threadIdx.x % 8;
        if (n >= left_n || 16 * w >= left_m) continue;
        const uint4 p = *reinterpret_cast<const uint4 *>(t + n * kBlock + 4 * piece(n, 4 * w));
        uint8_t *out = a.qt + (n0 + n) * a.qts + m0 + 16 * w;
        if (16 * w + 16 <= left_m) {
            *reinterpret_cast<uint4 *>(out) = p;
        } else {                           // bytes past the row's end are not ours
            const uint32_t b[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * w + i < left_m) out[i] = uint8_t(b[i / 4] >> (8 * (i % 4)));
        }
    }
}

// Rows that allow accesses of 16 bytes: a CTA walks tiles with the grid's
// stride, and the next tile's loads are on their way to shared memory while
// one is worked on.  A lane has N neighbouring columns (8 of 16 bits, 4 of
// 32) of R neighbouring rows, 64 values; it copies them itself and reads them
// from shared memory twice, for the maxima (16-bit values two at a time) and
// for the rounding, where a value is unpacked once for its row and its
// column.  Measured at 32768 x 6144 bf16 with the transpose: 138 us, 5.9 TB/s,
// with 8 warps; 190 with 16, whose 64 registers a thread spill.
// PER_ROW: 1 x 128 scales; otherwise one scale for the tile.
template <class T, bool PER_ROW>
__global__ void __launch_bounds__(kTileThreads, 2)
quantize_tile_kernel(const __grid_constant__ QuantArgs a, int tiles_n, int tiles_m) {
    constexpr int ST = kTileAhead + 1, N = Pack<T>::N, G = kBlock / N, R = kTileRows * G / 32;
    extern __shared__ __align__(16) uint8_t smem[];     // [ST][R][threads] of 16 bytes
    __shared__ __align__(16) uint32_t col_max[kTileWarps][kBlock];
    __shared__ float col_inv[kBlock];
    __shared__ __align__(16) uint8_t t[kBlock * kBlock];
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int r0 = warp * kTileRows + lane / G * R, c0 = lane % G * N;
    const T *const x = static_cast<const T *>(a.x);
    uint4 *const all = reinterpret_cast<uint4 *>(smem);
    // A tile's place, counted on by the grid's size instead of divided anew.
    struct Place {
        int m, n;
        __device__ __forceinline__ void next(int by_m, int by_n, int tiles_n) {
            m += by_m;
            n += by_n;
            if (n >= tiles_n) {
                n -= tiles_n;
                ++m;
            }
        }
    };
    const int by_m = int(gridDim.x) / tiles_n, by_n = int(gridDim.x) % tiles_n;
    Place now = {int(blockIdx.x) / tiles_n, int(blockIdx.x) % tiles_n}, ahead = now;
    auto fetch = [&](int stage) {
        const int64_t m = int64_t(ahead.m) * kBlock + r0, n = int64_t(ahead.n) * kBlock + c0;
        const T *from = x + m * a.xs + n;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool have = m + i < a.rows && n < a.cols;
            copy16_async(all + (stage * R + i) * kTileThreads + threadIdx.x, have ? from : x, have);
            from += a.xs;
        }
        copy_commit();
        ahead.next(by_m, by_n, tiles_n);
    };
    for (int i = 0; i < kTileAhead; ++i) fetch(i);
    int stage = ST - 1;
    for (; now.m < tiles_m; now.next(by_m, by_n, tiles_n)) {
        const int64_t tm = now.m;
        const int tn = now.n;
        const int64_t m0 = tm * kBlock, n0 = int64_t(tn) * kBlock;
        const int left_n = int(min(int64_t(kBlock), a.cols - n0));
        const int left_m = int(min(int64_t(kBlock), a.rows - m0));
        fetch(stage);
        copy_wait<kTileAhead>();
        stage = stage + 1 < ST ? stage + 1 : 0;
        const uint4 *mine = all + stage * R * kTileThreads + threadIdx.x;

        // Maxima: of the lane's columns over its rows, joined over the warp's
        // other rows where it holds two; of its rows over its columns.
        uint32_t col[4] = {0, 0, 0, 0};          // packed as the values are
        uint32_t row[R];                          // float bits
        {
            uint32_t two[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const uint4 v = mine[i * kTileThreads];
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                two[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    col[j] = Pack<T>::max_abs(col[j], u[j]);
                    two[i] = Pack<T>::max_abs(two[i], u[j]);
                }
            }
            if constexpr (N == 8) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    col[j] = Pack<T>::max_abs(col[j], __shfl_xor_sync(0xffffffffu, col[j], 16));
#pragma unroll
                for (int i = 0; i < R; i += 2) {  // rows i and i + 1 in one word
                    uint32_t m = Pack<T>::max_abs(__byte_perm(two[i], two[i + 1], 0x5410),
                                                  __byte_perm(two[i], two[i + 1], 0x7632));
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1)
                        m = Pack<T>::max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
                    m = Pack<T>::magnitude(m);
                    row[i] = Pack<T>::low(m);
                    row[i + 1] = Pack<T>::high(m);
                }
                if (lane < 16) *reinterpret_cast<uint4 *>(&col_max[warp][lane * 4]) =
                    make_uint4(col[0], col[1], col[2], col[3]);
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i)
                    row[i] = __reduce_max_sync(0xffffffffu, Pack<T>::magnitude(two[i]));
                *reinterpret_cast<uint4 *>(&col_max[warp][lane * 4]) = make_uint4(col[0], col[1], col[2], col[3]);
            }
        }
        // whether the tile holds an infinity: then each value is looked at
        bool inf_here = false;
#pragma unroll
        for (int i = 0; i < R; ++i) inf_here |= row[i] >= kInfBits;
        const bool infinite = __syncthreads_or(inf_here);
        uint32_t tile_sb = 127;
        if (!PER_ROW || a.qt != nullptr) {
            // column threadIdx.x of the tile (PER_ROW); all of them otherwise
            uint32_t m = 0;
            if (threadIdx.x < kBlock) {
                const int n = threadIdx.x;
                if (infinite) {
                    for (int r = 0; r < kBlock; ++r) {
                        const int i = r % kTileRows, th = r / kTileRows * 32 + i / R * G + n / N;
                        const T *v = reinterpret_cast<const T *>(all + (stage * R + i % R) * kTileThreads + th);
                        m = max(m, finite_bits(Elem<T>::to_float(v[n % N])));
                    }
                } else if constexpr (N == 8) {
                    uint32_t p = 0;
#pragma unroll
                    for (int w = 0; w < kTileWarps; ++w) p = Pack<T>::max_abs(p, col_max[w][n / 2]);
                    p = Pack<T>::magnitude(p);
                    m = n % 2 ? Pack<T>::high(p) : Pack<T>::low(p);
                } else {
#pragma unroll
                    for (int w = 0; w < kTileWarps; ++w) m = max(m, Pack<T>::magnitude(col_max[w][n]));
                }
                if (PER_ROW) {
                    const uint32_t sb = scale_byte(m);
                    col_inv[n] = inverse_scale(sb);
                    if (n < left_n) a.scales_t[(n0 + n) * a.sts + tm] = uint8_t(sb);
                } else {
                    m = __reduce_max_sync(0xffffffffu, m);
                    if (lane == 0) col_inv[warp] = __uint_as_float(m);
                }
            }
            __syncthreads();
            if (!PER_ROW) {
                m = 0;
#pragma unroll
                for (int w = 0; w < kBlock / 32; ++w) m = max(m, __float_as_uint(col_inv[w]));
                tile_sb = scale_byte(m);
                if (threadIdx.x == 0) {
                    if (a.q != nullptr) a.scales[tm * a.ss + tn] = uint8_t(tile_sb);
                    if (a.qt != nullptr) a.scales_t[tn * a.sts + tm] = uint8_t(tile_sb);
                }
            }
        }

        float inv[N];
#pragma unroll
        for (int j = 0; j < N; ++j) inv[j] = PER_ROW && a.qt != nullptr ? col_inv[c0 + j] : inverse_scale(tile_sb);
        uint8_t *q = a.q + (m0 + r0) * a.qs + n0 + c0, *scales = a.scales + (m0 + r0) * a.ss + tn;
#pragma unroll
        for (int k = 0; k < R; k += 4) {
            float v[4][N];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Pack<T>::unpack(mine[(k + i) * kTileThreads], v[i]);
                if (infinite) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < N; ++j) m = max(m, finite_bits(v[i][j]));
#pragma unroll
                    for (int o = G / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                    row[k + i] = m;
                    infinite_to_nan(v[i]);
                }
            }
            if (a.q != nullptr) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (r0 + k + i < left_m) {
                        const uint32_t sb = PER_ROW ? scale_byte(row[k + i]) : tile_sb;
                        if (PER_ROW && lane % G == 0) *scales = uint8_t(sb);
                        if (c0 < left_n) store_e4m3<N>(q, v[i], inverse_scale(sb));
                    }
                    q += a.qs;
                    scales += a.ss;
                }
            }
            if (a.qt != nullptr) {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    *reinterpret_cast<uint32_t *>(t + (c0 + j) * kBlock + 4 * piece(c0 + j, (r0 + k) / 4)) =
                        to_e4m3x4(v[0][j], v[1][j], v[2][j], v[3][j], inv[j]);
            }
        }
        if (a.qt != nullptr) {
            __syncthreads();
            store_transposed(a, t, m0, n0, left_m, left_n);
        }
        // No barrier here: what the next tile writes to col_max before its first
        // was read before this tile's second, and to t and col_inv after it.
    }
}

// Rows of any alignment: a tile a CTA, its values in registers, columns lane,
// lane + 32, ... of a row to a lane.  4099 x 5003 fp16 with 1 x 128 scales: 77 us, 12
// memory's time: single elements, no tile ahead of another.
template <class T, bool PER_ROW>
__global__ void __launch_bounds__(kTileThreads, 2)
quantize_any_tile_kernel(const __grid_constant__ QuantArgs a, int tiles_n) {
    __shared__ __align__(16) uint32_t col_max[kTileWarps][kBlock];
    __shared__ __align__(16) uint8_t t[kBlock * kBlock];
    grid_dependency();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t tm = blockIdx.x / tiles_n;
    const int tn = int(blockIdx.x % tiles_n);
    const int64_t m0 = tm * kBlock, n0 = int64_t(tn) * kBlock;
    const int left_n = int(min(int64_t(kBlock), a.cols - n0));
    const int left_m = int(min(int64_t(kBlock), a.rows - m0));
    const int r0 = warp * kTileRows;

    float v[kTileRows][4];
    const T *x = static_cast<const T *>(a.x) + (m0 + r0) * a.xs + n0;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) load4<T, false>(x + i * a.xs, lane, r0 + i < left_m ? left_n : 0, v[i]);

    uint32_t col[4] = {0, 0, 0, 0}, most = 0;
#pragma unroll
    for (int i = 0; i < kTileRows; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) col[j] = max(col[j], finite_bits(v[i][j]));
    most = max(max(col[0], col[1]), max(col[2], col[3]));
    uint32_t tile_sb = 127;
    if (PER_ROW) {
#pragma unroll
        for (int j = 0; j < 4; ++j) col_max[warp][lane + 32 * j] = col[j];
        __syncthreads();
    } else {
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) col_max[0][warp] = most;
        __syncthreads();
        tile_sb = scale_byte(__reduce_max_sync(0xffffffffu, lane < kTileWarps ? col_max[0][lane] : 0u));
        if (threadIdx.x == 0) {
            if (a.q != nullptr) a.scales[tm * a.ss + tn] = uint8_t(tile_sb);
            if (a.qt != nullptr) a.scales_t[tn * a.sts + tm] = uint8_t(tile_sb);
        }
    }
#pragma unroll
    for (int i = 0; i < kTileRows; ++i) {
        const uint32_t sb = PER_ROW ? row_scale(v[i]) : tile_sb;
        infinite_to_nan(v[i]);
        if (a.q == nullptr || r0 + i >= left_m) continue;
        const int64_t m = m0 + r0 + i;
        if (PER_ROW && lane == 0) a.scales[m * a.ss + tn] = uint8_t(sb);
        store4_e4m3<false>(a.q + m * a.qs + n0, lane, left_n, to_e4m3x4(v[i], inverse_scale(sb)));
    }
    if (a.qt == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = lane + 32 * j;
        uint32_t sb = tile_sb;
        if (PER_ROW) {
            uint32_t m = 0;
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) m = max(m, col_max[w][n]);
            sb = scale_byte(m);
            if (warp == 0 && n < left_n) a.scales_t[(n0 + n) * a.sts + tm] = uint8_t(sb);
        }
        const float inv = inverse_scale(sb);
#pragma unroll
        for (int k = 0; k < kTileRows; k += 4)
            *reinterpret_cast<uint32_t *>(t + n * kBlock + 4 * piece(n, (r0 + k) / 4)) =
                to_e4m3x4(v[k][j], v[k + 1][j], v[k + 2][j], v[k + 3][j], inv);
    }
    __syncthreads();
    store_transposed(a, t, m0, n0, left_m, left_n);
}

template <class T>
basp_status launch_tiles(const QuantArgs &a, bool per_row, bool vec16, cudaStream_t stream) {
    const int64_t blocks = ceil_div(a.cols, kBlock), tiles = ceil_div(a.rows, kBlock) * blocks;
    if (tiles > kMaxSide) return BASP_ERR_TOO_LARGE;
    if (!vec16) {
        auto kernel = per_row ? quantize_any_tile_kernel<T, true> : quantize_any_tile_kernel<T, false>;
        return launch(kernel, dim3(unsigned(tiles)), dim3(kTileThreads), 0, 1, stream, a, int(blocks));
    }
    constexpr size_t smem = size_t(kTileAhead + 1) * kBlock * kBlock * sizeof(T);
    auto tiles_of = [&](auto each_row) {
        constexpr auto kernel = quantize_tile_kernel<T, decltype(each_row)::value>;
        if (!allow_shared_memory<kernel, smem>()) return BASP_ERR_CUDA;
        const int64_t ctas = std::min(tiles, resident_ctas(kernel, kTileThreads, smem));
        return launch(kernel, dim3(unsigned(ctas)), dim3(kTileThreads), smem, 1, stream, a, int(blocks),
                      int(ceil_div(a.rows, kBlock)));
    };
    return per_row ? tiles_of(std::true_type()) : tiles_of(std::false_type());
}

template <class T, bool VEC>
basp_status launch_rows(const QuantArgs &a, cudaStream_t stream) {
    const int64_t groups = ceil_div(ceil_div(a.cols, kBlock), kRowBlocks);
    const int64_t ctas = ceil_div(a.rows * groups, kRowWarps);
    if (ctas > kMaxSide) return BASP_ERR_TOO_LARGE;
    return launch(quantize_rows_kernel<T, VEC>, dim3(unsigned(ctas)), dim3(kRowWarps * 32), 0, 1, stream, a,
                  int(groups));
}

template <class T>
basp_status launch_quantize(const QuantArgs &a, bool per_row, cudaStream_t stream) {
    if (!per_row || a.qt != nullptr)
        return launch_tiles<T>(a, per_row, vec16_ok(a.x, a.xs, a.cols, sizeof(T)), stream);
    return vec4_ok(a.x, a.xs, a.cols, sizeof(T)) ? launch_rows<T, true>(a, stream)
                                                 : launch_rows<T, false>(a, stream);
}

}  // namespace
}  // namespace basp_fp8

using namespace basp_fp8;

extern "C" basp_status basp_quantize_fp8(basp_dtype dtype, int64_t rows, int64_t cols, const void *x,
                                         int64_t x_stride, const basp_fp8_matrix *q,
                                         const basp_fp8_matrix *qt, cudaStream_t stream) {
    NvtxRange range("basp_quantize_fp8");
    basp_status st = BASP_OK;
    const int64_t esz = elem_size(dtype);
    if (esz == 0 || (q == nullptr && qt == nullptr)) return BASP_ERR_INVALID_ARG;
    if (!sides_ok(rows, cols, &st)) return st;
    if (q != nullptr && qt != nullptr && q->block_rows != qt->block_rows) return BASP_ERR_INVALID_ARG;
    Args args;
    args.matrix(x, rows, cols, x_stride, esz, false);
    if (q != nullptr) args.fp8(q, rows, cols, true);
    if (qt != nullptr) args.fp8(qt, cols, rows, true);
    st = args.status();
    if (st != BASP_OK || rows == 0 || cols == 0) return st;

    QuantArgs a = {};
    a.x = x; a.xs = x_stride; a.rows = rows; a.cols = int(cols);
    if (q != nullptr) {
        a.q = static_cast<uint8_t *>(q->data);
        a.scales = static_cast<uint8_t *>(q->scales);
        a.qs = q->pitch;
        a.ss = q->scale_pitch;
    }
    if (qt != nullptr) {
        a.qt = static_cast<uint8_t *>(qt->data);
        a.scales_t = static_cast<uint8_t *>(qt->scales);
        a.qts = qt->pitch;
        a.sts = qt->scale_pitch;
    }
    const bool per_row = (q != nullptr ? q : qt)->block_rows == 1;
    switch (dtype) {
        case BASP_DTYPE_BF16: return launch_quantize<__nv_bfloat16>(a, per_row, stream);
        case BASP_DTYPE_FP16: return launch_quantize<__half>(a, per_row, stream);
        default: return launch_quantize<float>(a, per_row, stream);
    }
}
