// attention.cu -- causal attention with a sliding window and sinks: forward,
// backward and one token over a cache (include/basp_attention.h).
//
// The calls' checks, what TMA needs to know of the tensors, and the plain form of a
// warp a row, for tensors that TMA cannot address (a sequence stride of 0 or below a
// head's length, strides of 2^40 bytes).
#include <algorithm>
#include <cmath>

#include "attention.cuh"

namespace basp_fp8 {
namespace {

__device__ unsigned long long g_timeouts;

constexpr int kRowWarps = 4;

enum { kForward, kDq, kDkv };

// Loops over a sequence step past its end by less than what is left of 32 bits.
constexpr int64_t kMaxLength = (int64_t(1) << 31) - 4096;

// A warp a row.
template <class T, int WHAT>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const __grid_constant__ AttentionArgs a) {
    grid_dependency();
    const int heads = WHAT == kDkv ? a.hkv : a.hq, len = WHAT == kDkv ? a.sk : a.sq;
    const int64_t rows = int64_t(a.batch) * heads * len;
    for (int64_t r = int64_t(blockIdx.x) * kRowWarps + threadIdx.x / 32; r < rows; r += int64_t(gridDim.x) * kRowWarps) {
        const int i = int(r % len), h = int(r / len % heads), b = int(r / len / heads);
        if constexpr (WHAT == kForward) forward_row<T, true>(a, b, h, i);
        if constexpr (WHAT == kDq) dq_row<T>(a, b, h, i);
        if constexpr (WHAT == kDkv) dkv_row<T>(a, b, h, i);
    }
}

template <class T, int WHAT> basp_status launch_rows(const AttentionArgs &a, cudaStream_t stream) {
    const int64_t rows = int64_t(a.batch) * (WHAT == kDkv ? int64_t(a.hkv) * a.sk : int64_t(a.hq) * a.sq);
    if (rows == 0) return BASP_OK;
    const int64_t ctas = std::min<int64_t>(ceil_div(rows, kRowWarps), 1 << 20);
    return launch(rows_kernel<T, WHAT>, dim3(unsigned(ctas)), dim3(kRowWarps * 32), 0, 1, stream, a);
}

// The statistics that the backward takes, of a tile of 128 queries a CTA: LANES lanes a
// row, 16 bytes each, and then a thread a row.  Memory is the bound; neighbouring CTAs have
// neighbouring heads, whose rows lie next to each other.
template <class T, int LANES>
__global__ void __launch_bounds__(256) stats_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int ROWS = 256 / LANES, PASSES = kTile / ROWS;
    __shared__ float sums[kTile];
    __shared__ float2 tops[kUnits<T> ? kTile : 1];            // largest |dO|, sum of |dO|
    grid_dependency();
    const int tiles = a.sq_pad / kTile, h = int(blockIdx.x % unsigned(a.hq)), tile = int(blockIdx.x / unsigned(a.hq) % unsigned(tiles));
    const int b = int(blockIdx.x / unsigned(a.hq) / unsigned(tiles)), head = b * a.hq + h, e = int(threadIdx.x % LANES) * 8;
    uint4 o[PASSES], g[PASSES];
    uint2 rest[PASSES];
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
        const int i = tile * kTile + x * ROWS + int(threadIdx.x) / LANES;
        const bool in = i < a.sq && e < a.d;
        o[x] = in ? *reinterpret_cast<const uint4 *>(row_of<const T>(a.o, b, i, h) + e) : make_uint4(0, 0, 0, 0);
        g[x] = in ? *reinterpret_cast<const uint4 *>(row_of<const T>(a.d_o, b, i, h) + e) : make_uint4(0, 0, 0, 0);
        rest[x] = in && a.rest.p != nullptr ? *reinterpret_cast<const uint2 *>(row_of<const int8_t>(a.rest, b, i, h) + e)
                                            : make_uint2(0, 0);
    }
    const int row = int(threadIdx.x), i = tile * kTile + row;
    const bool sees = row < kTile && i < a.sq && i + a.sk - a.sq >= 0;
    const float lse = sees ? a.lse[int64_t(head) * a.sq + i] * kLog2e : 0.f;
#pragma unroll
    for (int x = 0; x < PASSES; ++x) {
        float u[8], v[8], s = 0.f;
        Pack<T>::unpack(o[x], u);
        Pack<T>::unpack(g[x], v);
        if constexpr (kUnits<T>) {
            float top = 0.f, sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float y = fabsf(v[j]) < INFINITY ? fabsf(v[j]) : 0.f;
                top = fmaxf(top, y);
                sum += y;
            }
#pragma unroll
            for (int w = LANES / 2; w > 0; w >>= 1) {
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                sum += __shfl_xor_sync(0xffffffffu, sum, w);
            }
            if (threadIdx.x % LANES == 0) tops[x * ROWS + threadIdx.x / LANES] = make_float2(top, sum);
        }
        if (a.rest.p != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u[j] = with_lost<T>(u[j], int((j < 4 ? rest[x].x : rest[x].y) << (24 - j % 4 * 8)) >> 24);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(u[j], v[j], s);
#pragma unroll
        for (int w = LANES / 2; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        if (threadIdx.x % LANES == 0) sums[x * ROWS + threadIdx.x / LANES] = s;
    }
    __syncthreads();
    if (row >= kTile) return;
    const float s = sums[row];
    a.stats[int64_t(head) * a.sq_pad + i] = sees ? make_float2(lse, s) : make_float2(INFINITY, 0.f);
    // -lse / c and -D in parts of 16 bits: what is past their range is NaN, so that the rows
    // that meet it are made from the definition
    const float sign = a.scale < 0.f ? 1.f : -1.f;                // the other side of the product is negated
    bool past = false;
    float part[8], left = sees ? sign * lse / score_scale(a.scale) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float unit = fold_unit<T>(j % 4);
        if (j == 4) left = sees ? -s : 0.f;
        part[j] = unit == 0.f ? 0.f : Elem<T>::to_float(Elem<T>::from_float(left / unit));
        if (!(fabsf(part[j]) < INFINITY)) {
            part[j] = __uint_as_float(0x7fffffffu);
            past = true;
        }
        left -= part[j] * unit;
    }
    if constexpr (kUnits<T>) {
        const float2 own = sees ? tops[row] : make_float2(0.f, 0.f);
        const float top = warp_max(own.x), sum = warp_max(own.y), most = warp_max(sees && fabsf(s) < INFINITY ? fabsf(s) : 0.f);
        past = __any_sync(0xffffffffu, past && fabsf(lse) < INFINITY && fabsf(s) < INFINITY);
        a.unit[int64_t(head) * a.sq_pad + i] = unit_of(own.x);
        if (row % 32 == 0) a.peak[(int64_t(head) * a.sq_pad + i) / 32] = make_float4(top, sum, past ? INFINITY : most, 0.f);
    }
    uint8_t *to = reinterpret_cast<uint8_t *>(a.fold) + (int64_t(head) * a.sq_pad + tile * kTile) * 32 + fold_offset(row);
    const uint4 w = Pack<T>::pack(part);
    *reinterpret_cast<uint4 *>(to) = make_uint4(w.x, w.y, 0, 0);
    *reinterpret_cast<uint4 *>(to + kFoldPlane) = make_uint4(w.z, w.w, 0, 0);
}
template <class T> basp_status launch_stats(const AttentionArgs &a, cudaStream_t stream) {
    const int64_t ctas = int64_t(a.sq_pad / kTile) * a.batch * a.hq;
    if (ctas == 0) return BASP_OK;
    if (ctas > kMaxSide) return BASP_ERR_TOO_LARGE;
    return a.d <= 64 ? launch(stats_kernel<T, 8>, dim3(unsigned(ctas)), dim3(256), 0, 1, stream, a)
                     : launch(stats_kernel<T, 16>, dim3(unsigned(ctas)), dim3(256), 0, 1, stream, a);
}

// ---- host -----------------------------------------------------------------------

bool sizes_ok(const basp_attention_desc *d, basp_status *st) {
    *st = BASP_ERR_INVALID_ARG;
    if (d == nullptr || d->batch < 0 || d->q_len < 0 || d->k_len < 0 || d->q_heads < 0 || d->k_heads < 0 ||
        d->window < 0 || d->sinks < 0 || !(d->scale > -INFINITY && d->scale < INFINITY))
        return false;
    if (d->dtype != BASP_DTYPE_BF16 && d->dtype != BASP_DTYPE_FP16) return false;
    if (d->head_dim < 8 || d->head_dim > kMaxHeadDim || d->head_dim % 8) return false;
    if (d->k_heads == 0 ? d->q_heads != 0 : d->q_heads % d->k_heads != 0) {
        *st = BASP_ERR_DIVISIBILITY;
        return false;
    }
    *st = BASP_ERR_TOO_LARGE;
    for (int64_t n : {d->batch, d->q_heads, d->k_heads})
        if (n > kMaxSide) return false;
    for (int64_t n : {d->q_len, d->k_len})
        if (n > kMaxLength) return false;
    *st = BASP_OK;
    return true;
}

// Heads of all sequences fit a grid, and their rows the GPU's memory.
bool rows_ok(const basp_attention_desc *d) {
    const __int128 q = __int128(d->batch) * d->q_heads * d->q_len, k = __int128(d->batch) * d->k_heads * d->k_len;
    return q <= (int64_t(1) << 38) && k <= (int64_t(1) << 38) &&          // 2^38 rows are 4 TB
           d->batch * d->q_heads <= kMaxSide / 2 && d->batch * d->k_heads <= kMaxSide / 2;
}

// Checks of a call's tensors: each has len x heads rows of head_dim in each sequence.
class HeadArgs {
  public:
    explicit HeadArgs(const basp_attention_desc *d) : d_(d) {}
    void heads(const basp_heads *t, int64_t len, int64_t heads, bool out, int64_t esz = 2) {
        if (d_->batch == 0 || len == 0 || heads == 0) return;
        if (t == nullptr || t->data == nullptr || t->stride_batch < 0 || t->stride_seq < 0 || t->stride_head < 0)
            return fail(BASP_ERR_INVALID_ARG);
        if (uintptr_t(t->data) % uintptr_t(8 * esz) || t->stride_batch % 8 || t->stride_seq % 8 || t->stride_head % 8)
            return fail(BASP_ERR_ALIGNMENT);
        const int64_t n[3] = {d_->batch, len, heads};
        int64_t s[3] = {t->stride_batch, t->stride_seq, t->stride_head};
        __int128 last = 0;
        for (int i = 0; i < 3; ++i) {
            if (n[i] == 1) s[i] = 0;             // says nothing
            last += __int128(n[i] - 1) * s[i];
        }
        if (last > (int64_t(1) << 56)) return fail(BASP_ERR_TOO_LARGE);
        if (out && !apart(n, s)) return fail(BASP_ERR_ALIASING);
        args_.matrix(t->data, 1, int64_t(last) + d_->head_dim, 0, esz, out);
    }
    void vector(const void *p, int64_t n, int64_t esz, bool out, bool need = true) {
        args_.matrix(p, n > 0 ? 1 : 0, n, n, esz, out, need);
    }
    void fail(basp_status s) { args_.fail(s); }
    basp_status status() const { return args_.status(); }

  private:
    // Whether no two elements of an output share an address: from the smallest stride
    // outwards, each steps over all that the smaller ones reach.
    bool apart(const int64_t (&n)[3], const int64_t (&s)[3]) const {
        int order[3] = {0, 1, 2};
        std::sort(order, order + 3, [&](int x, int y) { return s[x] < s[y]; });
        __int128 reach = d_->head_dim;
        for (int i : order) {
            if (n[i] == 1) continue;
            if (s[i] < reach) return false;
            reach += __int128(n[i] - 1) * s[i];
        }
        return true;
    }
    const basp_attention_desc *d_;
    Args args_;
};

Heads heads_of(const basp_heads *t) {
    if (t == nullptr) return {};
    return {t->data, t->stride_batch, t->stride_seq, t->stride_head};
}

AttentionArgs args_of(const basp_attention_desc *d) {
    AttentionArgs a = {};
    a.batch = int(d->batch); a.sq = int(d->q_len); a.sk = int(d->k_len);
    a.hq = int(d->q_heads); a.hkv = int(d->k_heads); a.d = int(d->head_dim);
    a.group = d->k_heads > 0 ? int(d->q_heads / d->k_heads) : 1;
    const int64_t all = std::max<int64_t>(1, d->k_len);
    a.window = int(d->window == 0 ? all : std::min(d->window, all));
    a.sinks = int(std::min(d->sinks, d->k_len));
    a.scale = d->scale;
    return a;
}

// ---- TMA ------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) !=
                cudaSuccess || qr != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return EncodeFn(nullptr);
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Whether TMA can address the rows of a tensor of `len` x `heads` a sequence.
bool tma_ok(const AttentionArgs &a, const Heads &t, int len, int heads) {
    const int64_t most = (int64_t(1) << 39) - 1;          // 2^40 bytes
    return (len == 1 || (t.ss >= a.d && t.ss <= most)) && (heads == 1 || t.sh <= most) && (a.batch == 1 || t.sb <= most);
}

// Boxes of 64 values x `rows` rows; what is past a tensor's end reads zero.
bool encode(const AttentionArgs &a, const Heads &t, int len, int heads, int rows, CUtensorMap *out, int *head, int *batch) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    *head = heads > 1 && t.sh > 0;
    *batch = a.batch > 1 && t.sb > 0;
    const cuuint64_t dims[4] = {cuuint64_t(a.d), cuuint64_t(len), cuuint64_t(*head ? heads : 1), cuuint64_t(*batch ? a.batch : 1)};
    const cuuint64_t strides[3] = {cuuint64_t(len > 1 ? t.ss * 2 : kMaxHeadDim * 2), cuuint64_t(*head ? t.sh * 2 : kMaxHeadDim * 2),
                                   cuuint64_t(*batch ? t.sb * 2 : kMaxHeadDim * 2)};
    const cuuint32_t box[4] = {64, cuuint32_t(rows), 1, 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, t.p, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The count of waits that ran out, on the current device.
unsigned long long *timeouts_at() {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_timeouts) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return static_cast<unsigned long long *>(p);
}

bool encode_qkv(const AttentionArgs &a, HeadMaps *m) {
    m->timeouts = timeouts_at();
    return m->timeouts != nullptr && encode(a, a.q, a.sq, a.hq, kTile, &m->q, &m->q_head, &m->q_batch) &&
           encode(a, a.k, a.sk, a.hkv, kTile, &m->k, &m->k_head, &m->k_batch) &&
           encode(a, a.v, a.sk, a.hkv, kTile, &m->v, &m->v_head, &m->v_batch);
}

bool tiled(const AttentionArgs &a) {
    return a.sk > 0 && tma_ok(a, a.q, a.sq, a.hq) && tma_ok(a, a.k, a.sk, a.hkv) && tma_ok(a, a.v, a.sk, a.hkv);
}

template <class F> basp_status with_type(basp_dtype t, F &&f) {
    return t == BASP_DTYPE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

}  // namespace
}  // namespace basp_fp8

using namespace basp_fp8;

extern "C" basp_status basp_attention(const basp_attention_desc *desc, const basp_heads *q, const basp_heads *k,
                                      const basp_heads *v, const basp_heads *o, const basp_heads *o_rest,
                                      float *lse, cudaStream_t stream) {
    NvtxRange range("basp_attention");
    basp_status st;
    if (!sizes_ok(desc, &st)) return st;
    if (!rows_ok(desc)) return BASP_ERR_TOO_LARGE;
    HeadArgs args(desc);
    args.heads(q, desc->q_len, desc->q_heads, false);
    args.heads(k, desc->k_len, desc->k_heads, false);
    args.heads(v, desc->k_len, desc->k_heads, false);
    args.heads(o, desc->q_len, desc->q_heads, true);
    if (o_rest != nullptr) args.heads(o_rest, desc->q_len, desc->q_heads, true, 1);
    args.vector(lse, desc->batch * desc->q_heads * desc->q_len, 4, true, false);
    st = args.status();
    if (st != BASP_OK) return st;
    AttentionArgs a = args_of(desc);
    a.q = heads_of(q); a.k = heads_of(k); a.v = heads_of(v); a.o = heads_of(o);
    a.rest = heads_of(o_rest);
    a.lse = lse;
    if (a.batch == 0 || a.hq == 0 || a.sq == 0) return BASP_OK;
    if (tiled(a)) {
        HeadMaps m = {};
        if (!encode_qkv(a, &m)) return BASP_ERR_CUDA;
        return launch_attention_forward(a, m, desc->dtype == BASP_DTYPE_BF16, stream);
    }
    return with_type(desc->dtype, [&](auto t) { return launch_rows<decltype(t), kForward>(a, stream); });
}

// The statistics, their parts for the products and fp16's units: a multiple of 16 bytes.
static int64_t row_bytes(const AttentionArgs &a, basp_dtype t) {
    const int64_t rows = int64_t(a.batch) * a.hq * ceil_div(a.sq, kTile) * kTile;
    const int64_t tiles = int64_t(a.batch) * a.hkv * ceil_div(a.sk, kTile);
    return rows * (int64_t(sizeof(float2)) + 32) +
           (t == BASP_DTYPE_FP16 ? (rows + ceil_div(tiles, 4) * 4) * int64_t(sizeof(float)) + rows / 32 * int64_t(sizeof(float4)) : 0);
}

extern "C" int64_t basp_attention_backward_workspace(const basp_attention_desc *desc) {
    basp_status st;
    if (!sizes_ok(desc, &st) || !rows_ok(desc)) return 0;
    if (desc->batch == 0 || desc->q_heads == 0) return 0;
    const AttentionArgs a = args_of(desc);
    return row_bytes(a, desc->dtype) + key_split_bytes(a, key_split(a));
}

extern "C" basp_status basp_attention_backward(const basp_attention_desc *desc, const basp_heads *q,
                                               const basp_heads *k, const basp_heads *v, const basp_heads *o,
                                               const basp_heads *o_rest, const float *lse, const basp_heads *d_o, const basp_heads *dq,
                                               const basp_heads *dk, const basp_heads *dv, void *workspace,
                                               size_t workspace_bytes, cudaStream_t stream) {
    NvtxRange range("basp_attention_backward");
    basp_status st;
    if (!sizes_ok(desc, &st)) return st;
    if (!rows_ok(desc)) return BASP_ERR_TOO_LARGE;
    HeadArgs args(desc);
    args.heads(q, desc->q_len, desc->q_heads, false);
    args.heads(k, desc->k_len, desc->k_heads, false);
    args.heads(v, desc->k_len, desc->k_heads, false);
    args.heads(o, desc->q_len, desc->q_heads, false);
    if (o_rest != nullptr) args.heads(o_rest, desc->q_len, desc->q_heads, false, 1);
    args.heads(d_o, desc->q_len, desc->q_heads, false);
    args.heads(dq, desc->q_len, desc->q_heads, true);
    args.heads(dk, desc->k_len, desc->k_heads, true);
    args.heads(dv, desc->k_len, desc->k_heads, true);
    args.vector(lse, desc->batch * desc->q_heads * desc->q_len, 4, false);
    const int64_t need = basp_attention_backward_workspace(desc);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < size_t(need)) args.fail(BASP_ERR_WORKSPACE);
        else if (uintptr_t(workspace) % 16) args.fail(BASP_ERR_ALIGNMENT);
        else args.vector(workspace, need, 1, true);
    }
    st = args.status();
    if (st != BASP_OK) return st;
    AttentionArgs a = args_of(desc);
    a.q = heads_of(q); a.k = heads_of(k); a.v = heads_of(v); a.o = heads_of(o); a.d_o = heads_of(d_o);
    a.dq = heads_of(dq); a.dk = heads_of(dk); a.dv = heads_of(dv);
    a.rest = heads_of(o_rest);
    a.lse = const_cast<float *>(lse);
    a.sq_pad = int(ceil_div(a.sq, kTile) * kTile);
    a.stats = static_cast<float2 *>(workspace);
    const int64_t rows = int64_t(a.batch) * a.hq * a.sq_pad;
    a.fold = reinterpret_cast<uint16_t *>(a.stats + rows);
    a.unit = reinterpret_cast<float *>(a.fold + rows * 16);
    a.peak = reinterpret_cast<float4 *>(a.unit + rows);
    a.v_peak = reinterpret_cast<float *>(a.peak + rows / 32);
    // lse / c of the smallest scales is past 32 bits
    const bool tiles = a.batch > 0 && a.hq > 0 && a.sq > 0 && tiled(a) && tma_ok(a, a.d_o, a.sq, a.hq) &&
                       (a.scale == 0.f || std::fabs(a.scale) >= 0x1p-64f);
    HeadMaps m = {};
    if (tiles && (!encode_qkv(a, &m) || !encode(a, a.d_o, a.sq, a.hq, kTile, &m.d_o, &m.do_head, &m.do_batch)))
        return BASP_ERR_CUDA;
    return with_type(desc->dtype, [&](auto t) {
        using T = decltype(t);
        basp_status s = launch_stats<T>(a, stream);
        if (s == BASP_OK && tiles) {
            KeySplit split = key_split(a);
            split.past = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(workspace) + row_bytes(a, desc->dtype));
            split.partial = reinterpret_cast<float *>(split.past + ceil_div(key_split_parts(a, split), 4) * 4);
            return launch_attention_backward(a, m, split, desc->dtype == BASP_DTYPE_BF16, stream);
        }
        if (s == BASP_OK) s = launch_rows<T, kDq>(a, stream);
        if (s == BASP_OK) s = launch_rows<T, kDkv>(a, stream);
        return s;
    });
}

extern "C" int64_t basp_attention_decode_workspace(const basp_attention_desc *desc) {
    basp_status st;
    if (!sizes_ok(desc, &st) || !rows_ok(desc) || desc->batch == 0 || desc->q_heads == 0) return 0;
    return decode_workspace(args_of(desc));
}

extern "C" basp_status basp_attention_decode(const basp_attention_desc *desc, const basp_heads *q,
                                             const basp_heads *k, const basp_heads *v, const int32_t *lengths,
                                             const basp_heads *o, void *workspace, size_t workspace_bytes,
                                             cudaStream_t stream) {
    NvtxRange range("basp_attention_decode");
    basp_status st;
    if (!sizes_ok(desc, &st)) return st;
    if (desc->q_len != 1) return BASP_ERR_INVALID_ARG;
    if (!rows_ok(desc) || !decode_fits(args_of(desc))) return BASP_ERR_TOO_LARGE;
    HeadArgs args(desc);
    args.heads(q, 1, desc->q_heads, false);
    args.heads(k, desc->k_len, desc->k_heads, false);
    args.heads(v, desc->k_len, desc->k_heads, false);
    args.heads(o, 1, desc->q_heads, true);
    args.vector(lengths, desc->batch, 4, false);
    const int64_t need = basp_attention_decode_workspace(desc);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < size_t(need)) args.fail(BASP_ERR_WORKSPACE);
        else if (uintptr_t(workspace) % 16) args.fail(BASP_ERR_ALIGNMENT);
        else args.vector(workspace, need, 1, true);
    }
    st = args.status();
    if (st != BASP_OK || desc->batch == 0 || desc->q_heads == 0) return st;
    AttentionArgs a = args_of(desc);
    a.q = heads_of(q); a.k = heads_of(k); a.v = heads_of(v); a.o = heads_of(o);
    return launch_attention_decode(a, lengths, workspace, desc->dtype == BASP_DTYPE_BF16, stream);
}

extern "C" basp_status basp_attention_timeouts(unsigned long long *count) {
    if (count == nullptr) return BASP_ERR_INVALID_ARG;
    const unsigned long long zero = 0;
    if (cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpyFromSymbol(count, g_timeouts, sizeof(*count)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_timeouts, &zero, sizeof(zero)) != cudaSuccess) {
        cudaGetLastError();
        return BASP_ERR_CUDA;
    }
    return BASP_OK;
}
