// quantize.cu -- 16- and 32-bit matrices to e4m3 with a power-of-two scale for
// each 1 x 128 or 128 x 128 block, and the same for the transpose
// (basp_quantize_fp8).
//
// Each value is read once whatever is asked for: the bound is memory (3 bytes
// a value for a 16-bit matrix, 4 with the transpose).  Rows alone need no
// tile: a warp owns 128-blocks, four values a lane.  The transpose and
// 128 x 128 scales work on a 128 x 128 tile a CTA: warp w holds rows 16w to
// 16w+15 in registers (64 values a lane), so a row's maximum is one warp
// reduction, a column's maximum is a maximum over the lane's own 16 values
// joined across the eight warps in shared memory, and the 16 values that a
// lane holds of a column are 16 consecutive bytes of the transpose, which go
// through shared memory to leave as 128-byte rows.
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

// Warp units are groups of kRowBlocks neighbouring blocks of one row.
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
        const uint32_t sb = scale_byte(__reduce_max_sync(0xffffffffu, max_bits4(v[i])));
        store4_e4m3<VEC>(a.q + row * a.qs + c, lane, int(a.cols - c), to_e4m3x4(v[i], inverse_scale(sb)));
        if (lane == 0) a.scales[row * a.ss + b0 + i] = uint8_t(sb);
    }
}

// ---- tiles ----------------------------------------------------------------

constexpr int kTileWarps = 8;
constexpr int kTileRows = kBlock / kTileWarps;      // rows a warp

// Where 16-byte piece `w` of transposed row n sits in its 128 bytes of shared
// memory: eight neighbouring lanes, whose n differ by 1 or by 4, hit eight
// different pieces, so the 16-byte stores and loads are free of conflicts.
__device__ __forceinline__ int piece(int n, int w) { return w ^ ((n ^ (n >> 2)) & 7); }

// PER_ROW: 1 x 128 scales; otherwise one scale for the tile.
template <class T, bool VEC, bool PER_ROW>
__global__ void __launch_bounds__(kTileWarps * 32)
quantize_tile_kernel(const __grid_constant__ QuantArgs a, int tiles_n) {
    __shared__ uint32_t col_max[kTileWarps][kBlock];
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
    for (int i = 0; i < kTileRows; ++i) {
        if (r0 + i < left_m) {
            load4<T, VEC>(x + i * a.xs, lane, left_n, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = 0.f;
        }
    }

    uint32_t tile_sb = 127;
    if (!PER_ROW) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) m = max(m, max_bits4(v[i]));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) col_max[warp][0] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTileWarps; ++w) m = max(m, col_max[w][0]);
        tile_sb = scale_byte(m);
        if (threadIdx.x == 0) {
            if (a.q != nullptr) a.scales[tm * a.ss + tn] = uint8_t(tile_sb);
            if (a.qt != nullptr) a.scales_t[tn * a.sts + tm] = uint8_t(tile_sb);
        }
    }

    if (a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < kTileRows; ++i) {
            if (r0 + i >= left_m) break;
            const int64_t m = m0 + r0 + i;
            uint32_t sb = tile_sb;
            if (PER_ROW) {
                sb = scale_byte(__reduce_max_sync(0xffffffffu, max_bits4(v[i])));
                if (lane == 0) a.scales[m * a.ss + tn] = uint8_t(sb);
            }
            store4_e4m3<VEC>(a.q + m * a.qs + n0, lane, left_n, to_e4m3x4(v[i], inverse_scale(sb)));
        }
    }
    if (a.qt == nullptr) return;

    uint32_t sb[4] = {tile_sb, tile_sb, tile_sb, tile_sb};
    if (PER_ROW) {
        uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kTileRows; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = max(m[j], finite_bits(v[i][j]));
#pragma unroll
        for (int j = 0; j < 4; ++j) col_max[warp][lane_col<VEC>(lane, j)] = m[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = lane_col<VEC>(lane, j);
#pragma unroll
            for (int w = 0; w < kTileWarps; ++w) m[j] = max(m[j], col_max[w][n]);
            sb[j] = scale_byte(m[j]);
            if (warp == 0 && n < left_n) a.scales_t[(n0 + n) * a.sts + tm] = uint8_t(sb[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = lane_col<VEC>(lane, j);
        const float inv = inverse_scale(sb[j]);
        uint32_t p[kTileRows / 4];
#pragma unroll
        for (int k = 0; k < kTileRows / 4; ++k) {
            const float c[4] = {v[4 * k][j], v[4 * k + 1][j], v[4 * k + 2][j], v[4 * k + 3][j]};
            p[k] = to_e4m3x4(c, inv);
        }
        *reinterpret_cast<uint4 *>(t + n * kBlock + 16 * piece(n, warp)) = make_uint4(p[0], p[1], p[2], p[3]);
    }
    __syncthreads();
    // 16 bytes a thread, eight threads a transposed row, four rounds
#pragma unroll
    for (int k = 0; k < kBlock * kBlock / (16 * kTileWarps * 32); ++k) {
        const int n = k * (kTileWarps * 4) + int(threadIdx.x) / 8, w = threadIdx.x % 8;
        if (n >= left_n || 16 * w >= left_m) continue;
        const uint4 p = *reinterpret_cast<const uint4 *>(t + n * kBlock + 16 * piece(n, w));
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

template <class T, bool VEC>
basp_status launch_quantize(const QuantArgs &a, bool per_row, cudaStream_t stream) {
    const int64_t blocks = ceil_div(a.cols, kBlock);
    if (per_row && a.qt == nullptr) {
        const int64_t groups = ceil_div(blocks, kRowBlocks);
        const int64_t ctas = ceil_div(a.rows * groups, kRowWarps);
        if (ctas > kMaxSide) return BASP_ERR_TOO_LARGE;
        return launch(quantize_rows_kernel<T, VEC>, dim3(unsigned(ctas)), dim3(kRowWarps * 32), 0, 1, stream,
                      a, int(groups));
    }
    const int64_t tiles = ceil_div(a.rows, kBlock) * blocks;
    if (tiles > kMaxSide) return BASP_ERR_TOO_LARGE;
    const dim3 grid(static_cast<unsigned>(tiles)), block(kTileWarps * 32);
    if (per_row)
        return launch(quantize_tile_kernel<T, VEC, true>, grid, block, 0, 1, stream, a, int(blocks));
    return launch(quantize_tile_kernel<T, VEC, false>, grid, block, 0, 1, stream, a, int(blocks));
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
    const bool vec = vec4_ok(x, x_stride, cols, esz);
    switch (dtype) {
        case BASP_DTYPE_BF16:
            return vec ? launch_quantize<__nv_bfloat16, true>(a, per_row, stream)
                       : launch_quantize<__nv_bfloat16, false>(a, per_row, stream);
        case BASP_DTYPE_FP16:
            return vec ? launch_quantize<__half, true>(a, per_row, stream)
                       : launch_quantize<__half, false>(a, per_row, stream);
        default:
            return vec ? launch_quantize<float, true>(a, per_row, stream)
                       : launch_quantize<float, false>(a, per_row, stream);
    }
}
