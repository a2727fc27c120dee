// attention_common.cuh -- what the attention kernels share: which keys a query
// sees, the tensors as kernels take them, and the plain form, row by row.
#pragma once

#include "basp_attention.h"
#include "fp8_common.cuh"
#include "tcgen05.cuh"

namespace basp_fp8 {

constexpr int kMaxHeadDim = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct Heads {
    void *p;
    int64_t sb, ss, sh;
};

template <class T> __device__ __forceinline__ T *row_of(const Heads &t, int64_t b, int64_t s, int64_t h) {
    return static_cast<T *>(t.p) + b * t.sb + s * t.ss + h * t.sh;
}

struct AttentionArgs {
    Heads q, k, v, o, rest, d_o, dq, dk, dv;     // rest: what o lost in its rounding (lost_of), or none
    float *lse;                          // [batch][Hq][Sq]
    // for the backward: (lse log2(e), D) of each query, [batch][Hq][sq_pad]; of one that
    // does not exist, or sees nothing: (infinity, 0)
    float2 *stats;
    uint16_t *fold;                      // the same as parts of a product, two planes a tile of queries
    // fp16: unit_of each query's dO [batch][Hq][sq_pad]; of 32 queries the largest |dO|, sum of |dO|
    // and |D| (infinite where a part of lse or D of one is past the type's range); of each tile of
    // keys the largest |v|
    float *unit;
    float4 *peak;
    float *v_peak;
    int batch, sq, sk, sq_pad, hq, hkv, d, group;
    int window, sinks;                   // window: sk where all is visible
    float scale;
};

// ---- tiles of 128 queries and keys ---------------------------------------------------

constexpr int kTile = 128;
constexpr int kBox = kTile * 128;        // bytes of a box of 128 rows x 64 values

// Key tiles that any of the queries [r0, r0 + 128) sees: [0, first) and [low, high).
struct KeyTiles {
    int first, low, high;
    __device__ __forceinline__ bool has(int j) const { return j < first || (j >= low && j < high); }
    __device__ __forceinline__ int count() const { return first + high - low; }
    __device__ __forceinline__ int begin() const { return first > 0 ? 0 : low; }
    // the one after j; `high` where there is none
    __device__ __forceinline__ int next(int j) const { return j + 1 == first ? low : j + 1; }
};
__device__ __forceinline__ KeyTiles key_tiles(const AttentionArgs &a, int r0) {
    const int p1 = min(r0 + kTile, a.sq) - 1 + a.sk - a.sq;
    if (r0 >= a.sq || p1 < 0) return {0, 0, 0};
    const int low = max(0, max(0, r0 + a.sk - a.sq) - a.window + 1) / kTile;
    const int first_end = min(a.sinks, max(0, p1 - a.window + 1));
    return {min((first_end + kTile - 1) / kTile, low), low, p1 / kTile + 1};
}

// Key j is seen by the positions [j, last position].
__host__ __device__ __forceinline__ int last_position(const AttentionArgs &a, int j) {
    const int64_t last = int64_t(j) + a.window - 1;
    return j < a.sinks || last >= a.sk ? a.sk - 1 : int(last);
}

// Query tiles that see any of the keys [k0, k0 + 128): [low, high).
struct QueryTiles {
    int low, high;
};
__host__ __device__ __forceinline__ QueryTiles query_tiles(const AttentionArgs &a, int k0) {
    const int shift = a.sk - a.sq, k1 = (a.sk - k0 < kTile ? a.sk : k0 + kTile) - 1;
    const int last = (k0 < a.sinks ? a.sk - 1 : last_position(a, k1)) - shift, first = k0 > shift ? k0 - shift : 0;
    if (last < first) return {0, 0};
    return {first / kTile, last / kTile + 1};
}

// A CTA's item in round r of the grid: rounds go to and fro, so that items of falling work
// come out even.  Past the last one where it is not below their number.
__device__ __forceinline__ int item_of(int r) {
    return r * int(gridDim.x) + (r % 2 ? int(gridDim.x) - 1 - int(blockIdx.x) : int(blockIdx.x));
}

// Bits 0 to n of a word.
__device__ __forceinline__ uint32_t bits_to(int n) { return n < 0 ? 0u : n >= 31 ? 0xffffffffu : (2u << n) - 1u; }

// What scores are multiplied by before 2^x (a negative scale negates one operand); a scale
// of 0 leaves all scores alike.
__device__ __forceinline__ float score_scale(float scale) { return fmaxf(fabsf(scale) * kLog2e, 0x1p-64f); }

// 8 values of K for each of 128 rows, as 16 bytes x 8 rows next to each other: a plane.  A
// tile of queries has one of its lse and one of its D.
constexpr int kFoldPlane = kTile * 16;
__host__ __device__ __forceinline__ constexpr int fold_offset(int row) { return row * 16; }
// Part j of lse / c, or of D, is multiplied by 1 / fold_unit(j) and the other side of the
// product has fold_unit(j) instead of one.  fp16's range is small at both ends: the first
// part may be 64 x 65504, and the third is exact to 2^-41.
template <class T> __host__ __device__ __forceinline__ constexpr float fold_unit(int j) {
    if (!std::is_same_v<T, __half>) return 1.f;
    return j == 0 ? 0x1p6f : j == 1 ? 0x1p-5f : j == 2 ? 0x1p-16f : 0.f;
}

// fp16 is exact to 2^-11 from 2^-14 on only, and small gradients have dS far below that (16384
// keys have P = 2^-14 on average).  So P and dS are rounded in units of their own: P of the dkv
// kernel in 2^-10 (its scores' errors may make it larger than one), and dS in a power of two near
// the largest |dO| of the query (dq), or of all queries that a CTA visits (dk), which leaves a
// factor of 2^15 above |dO| to dP = dO V^T.
template <class T> constexpr bool kUnits = std::is_same_v<T, __half>;
constexpr float kProbabilityExponent = 10.f, kProbabilityUnit = 0x1p-10f;
// 2^-e of the finite m in [2^e, 2^(e + 1)), 1 of zero; and 1 / unit.
__device__ __forceinline__ float unit_of(float m) {
    return m > 0.f ? __uint_as_float((254u << 23) - (__float_as_uint(m) & 0x7f800000u)) : 1.f;
}
__device__ __forceinline__ float over_unit(float unit) { return __uint_as_float((254u << 23) - __float_as_uint(unit)); }

// |dP - D| is at most sum |dO| max |v| + |D|: whether that is past fp16 in the unit, a factor of four
// kept for P.  Of finite values: where dS is no number itself, this does not say so.
__device__ __forceinline__ bool past_half(float unit, float sum, float v, float d) {
    return unit * fmaf(sum, v, d) > 65504.f / 4;
}
template <class T> __device__ __forceinline__ float finite_peak(uint4 x) {
    float f[8], top = 0.f;
    Pack<T>::unpack(x, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]) < INFINITY ? fabsf(f[j]) : 0.f);
    return top;
}

// A wait on one of the CTA's barriers, with a limit.
constexpr uint64_t kAttentionWaitNs = 2000000000ull;
struct AttentionWaiter {
    volatile int *abort;                 // shared by the CTA
    unsigned long long *timeouts;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, bool give_up_early = true) const {
        if (mbar_try_wait<false>(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait<false>(bar, parity)) {
            if (give_up_early && *abort) return false;
            if (global_ns() - t0 > kAttentionWaitNs) {
                if (!*abort) atomicAdd(timeouts, 1ull);
                *abort = 1;
                return false;
            }
        }
        return true;
    }
};

// A ring's place and the parity of its turn.
template <int N> struct Turn {
    uint32_t at = 0, turn = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            turn ^= 1;
        }
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest of three, a NaN not counted.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <class T> __device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __half2 p = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
}
template <class T> __device__ __forceinline__ float2 unpack_pair(uint32_t v) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&v));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

// The query at position p sees keys [0, first_end) and [last, p].
struct Sees {
    int first_end, last;
};
__device__ __forceinline__ Sees keys_of(const AttentionArgs &a, int p) {
    const int low = p < 0 ? 0 : max(0, p - a.window + 1);
    return {min(a.sinks, low), low};
}
// ---- the plain form -----------------------------------------------------------------
//
// A warp computes one row from its definition, reading nothing but what the row
// sees: lanes hold a key (or a query) each for the products, then four elements of
// the row each for the sums.

// What x lost when it was rounded to `rounded` of type T, in 256ths of its last place, cut: the
// difference of their 32-bit patterns, whose sign is the same, is in the bits that T does not
// have.  (A value that became 0, or one of fp16's subnormals, has more: as much as fits.)  And x
// from both, to 2^-17 (fp16: 2^-20) of itself; what is no number stays.
template <class T> constexpr int kLostShift = std::is_same_v<T, __half> ? 5 : 8;
template <class T> __device__ __forceinline__ int lost_of(float x, float rounded) {
    return int(__float_as_uint(x) - __float_as_uint(rounded)) >> kLostShift<T>;
}
template <class T> __device__ __forceinline__ float with_lost(float rounded, int lost) {
    const uint32_t add = (uint32_t(lost) << kLostShift<T>) + (1u << (kLostShift<T> - 1));
    return fabsf(rounded) < INFINITY ? __uint_as_float(__float_as_uint(rounded) + add) : rounded;
}
// Four of them as bytes, each at most 127 and at least -128.
__device__ __forceinline__ uint32_t lost_bytes(int a, int b, int c, int d) {
    uint32_t high, all;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(high) : "r"(d), "r"(c), "r"(0));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(all) : "r"(b), "r"(a), "r"(high));
    return all;
}

template <class T> __device__ __forceinline__ float row_dot(const T *x, const T *y, int d) {
    float s = 0.f;
    for (int e = 0; e < d; e += 8) {
        float f[8], g[8];
        Pack<T>::unpack(*reinterpret_cast<const uint4 *>(x + e), f);
        Pack<T>::unpack(*reinterpret_cast<const uint4 *>(y + e), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(f[j], g[j], s);
    }
    return s;
}

template <class T> __device__ __forceinline__ void row_add(float (&sum)[4], float p, const T *row, int d, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < d) sum[j] = fmaf(p, Elem<T>::to_float(row[lane + 32 * j]), sum[j]);
}

template <class T> __device__ __forceinline__ void row_store(T *row, const float (&v)[4], int d, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < d) row[lane + 32 * j] = Elem<T>::from_float(v[j]);
}

// Calls f(j, have) for 32 keys at a time of [0, first_end) and [low, end), until it says
// that the rest makes no difference; `have`: whether this lane's key exists.
template <class F> __device__ __forceinline__ bool each_keys(int first_end, int low, int end, int lane, F &&f) {
    for (int j0 = 0; j0 < first_end; j0 += 32)
        if (!f(j0 + lane, j0 + lane < first_end)) return false;
    for (int j0 = low; j0 < end; j0 += 32)
        if (!f(j0 + lane, j0 + lane < end)) return false;
    return true;
}

// Whether the warp's whole row is NaN, which no more addition changes.
__device__ __forceinline__ bool row_lost(const float (&v)[4], int d, int lane) {
    bool lost = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) lost = lost && (lane + 32 * j >= d || v[j] != v[j]);
    return __all_sync(0xffffffffu, lost);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = v > w || v != v ? v : w;                 // a NaN stays
    }
    return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// o of query i, and with LSE its lse.
template <class T, bool LSE>
__device__ __noinline__ void forward_row(const AttentionArgs &a, int b, int h, int i) {
    const int lane = threadIdx.x % 32, p = i + a.sk - a.sq, kh = h / a.group;
    const Sees see = keys_of(a, p);
    const T *q = row_of<const T>(a.q, b, i, h);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    each_keys(see.first_end, see.last, p + 1, lane, [&](int j, bool have) {
        const float s = have ? a.scale * row_dot(q, row_of<const T>(a.k, b, j, kh), a.d) : -INFINITY;
        const float top = warp_max(s), next = m > top || m != m ? m : top;
        // scores of minus infinity weigh nothing, also before the first that is more
        const float w = have && next != -INFINITY ? expf(s - next) : 0.f, old = m == -INFINITY && l == 0.f ? 0.f : expf(m - next);
        l = l * old + warp_add(w);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= old;
        m = next;
        for (int x = 0; x < 32; ++x) {
            const int jx = __shfl_sync(0xffffffffu, j, x);
            const float wx = __shfl_sync(0xffffffffu, w, x);
            if (__shfl_sync(0xffffffffu, int(have), x)) row_add(o, wx, row_of<const T>(a.v, b, jx, kh), a.d, lane);
        }
        return (LSE && l == l) || !row_lost(o, a.d, lane);
    });
    const bool any = p >= 0;                         // whoever sees anything sees itself
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = any ? o[e] / l : 0.f;
    row_store(row_of<T>(a.o, b, i, h), o, a.d, lane);
    if (a.rest.p != nullptr) {
        int8_t *rest = row_of<int8_t>(a.rest, b, i, h);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (lane + 32 * e < a.d)
                rest[lane + 32 * e] = int8_t(max(-128, min(127, lost_of<T>(o[e], Elem<T>::to_float(Elem<T>::from_float(o[e]))))));
    }
    if (LSE && a.lse != nullptr && lane == 0)
        a.lse[(int64_t(b) * a.hq + h) * a.sq + i] = any ? m + logf(l) : -INFINITY;
}

// dq of query i.
template <class T>
__device__ __noinline__ void dq_row(const AttentionArgs &a, int b, int h, int i) {
    const int lane = threadIdx.x % 32, p = i + a.sk - a.sq, kh = h / a.group;
    const Sees see = keys_of(a, p);
    const T *q = row_of<const T>(a.q, b, i, h), *d_o = row_of<const T>(a.d_o, b, i, h);
    const float lse = a.lse[(int64_t(b) * a.hq + h) * a.sq + i];
    const float delta = a.stats[(int64_t(b) * a.hq + h) * a.sq_pad + i].y;
    float dq[4] = {0.f, 0.f, 0.f, 0.f};
    each_keys(see.first_end, see.last, p + 1, lane, [&](int j, bool have) {
        float ds = 0.f;
        if (have) {
            const float w = expf(a.scale * row_dot(q, row_of<const T>(a.k, b, j, kh), a.d) - lse);
            ds = w * (row_dot(d_o, row_of<const T>(a.v, b, j, kh), a.d) - delta) * a.scale;
        }
        for (int x = 0; x < 32; ++x) {
            const int jx = __shfl_sync(0xffffffffu, j, x);
            const float dx = __shfl_sync(0xffffffffu, ds, x);
            if (__shfl_sync(0xffffffffu, int(have), x)) row_add(dq, dx, row_of<const T>(a.k, b, jx, kh), a.d, lane);
        }
        return !row_lost(dq, a.d, lane);
    });
    row_store(row_of<T>(a.dq, b, i, h), dq, a.d, lane);
}

// dk and dv of key j, over all query heads that share it.
template <class T>
__device__ __noinline__ void dkv_row(const AttentionArgs &a, int b, int kh, int j) {
    const int lane = threadIdx.x % 32, shift = a.sk - a.sq;
    const T *k = row_of<const T>(a.k, b, j, kh), *v = row_of<const T>(a.v, b, j, kh);
    const int i0 = max(0, j - shift), i1 = last_position(a, j) - shift + 1;
    float dk[4] = {0.f, 0.f, 0.f, 0.f}, dv[4] = {0.f, 0.f, 0.f, 0.f};
    bool go_on = true;
    for (int h = kh * a.group; h < (kh + 1) * a.group && go_on; ++h) {
        const float *lse = a.lse + (int64_t(b) * a.hq + h) * a.sq;
        const float2 *stats = a.stats + (int64_t(b) * a.hq + h) * a.sq_pad;
        go_on = each_keys(0, i0, i1, lane, [&](int i, bool have) {
            float w = 0.f, ds = 0.f;
            if (have) {
                w = expf(a.scale * row_dot(k, row_of<const T>(a.q, b, i, h), a.d) - lse[i]);
                ds = w * (row_dot(v, row_of<const T>(a.d_o, b, i, h), a.d) - stats[i].y) * a.scale;
            }
            for (int x = 0; x < 32; ++x) {
                const int ix = __shfl_sync(0xffffffffu, i, x);
                const float wx = __shfl_sync(0xffffffffu, w, x), dx = __shfl_sync(0xffffffffu, ds, x);
                if (__shfl_sync(0xffffffffu, int(have), x)) {
                    row_add(dv, wx, row_of<const T>(a.d_o, b, ix, h), a.d, lane);
                    row_add(dk, dx, row_of<const T>(a.q, b, ix, h), a.d, lane);
                }
            }
            return !(row_lost(dk, a.d, lane) && row_lost(dv, a.d, lane));
        });
    }
    row_store(row_of<T>(a.dk, b, j, kh), dk, a.d, lane);
    row_store(row_of<T>(a.dv, b, j, kh), dv, a.d, lane);
}

// ---- rows of tiles that came out infinite or NaN -------------------------------------
//
// A masked pair has P = 0 and dS = 0, but 0 times an infinite or NaN value is NaN.  Only a
// row with such a value among what its tiles hold and it does not see is computed again, and in
// fp16 one that met a dS, lse or D past the type's range: where what a row sees is no number
// itself, the tiles' answer is the definition's.  So a batch that has become NaN costs the search
// through the ends of its tiles, a row at a time, and no walk over all that a row sees.

// Whether a row holds a value that is infinite or NaN.
template <class T> __device__ __forceinline__ bool any_in_row(const T *row, int d) {
    bool bad = false;
    for (int e = 0; e < d; e += 8) {
        float f[8];
        Pack<T>::unpack(*reinterpret_cast<const uint4 *>(row + e), f);
#pragma unroll
        for (int j = 0; j < 8; ++j) bad = bad || !(fabsf(f[j]) < INFINITY);
    }
    return bad;
}
// Whether rows [s0, s1) of head h do.
template <class T>
__device__ __forceinline__ bool any_not_finite(const Heads &t, int b, int h, int s0, int s1, int d, int lane) {
    for (int s = s0; s < s1; s += 32)
        if (__any_sync(0xffffffffu, s + lane < s1 && any_in_row<T>(row_of<const T>(t, b, s + lane, h), d))) return true;
    return false;
}

// Of the query at position p in the tile of queries from r0: the keys of `t`.
template <class T>
__device__ __noinline__ bool masked_keys_not_finite(const AttentionArgs &a, const Heads &t, int b, int kh, int r0, int p) {
    const int lane = threadIdx.x % 32;
    const KeyTiles tiles = key_tiles(a, r0);
    const Sees see = keys_of(a, p);
    const int low = tiles.low * kTile, high = min(tiles.high * kTile, a.sk);
    return any_not_finite<T>(t, b, kh, see.first_end, min(tiles.first * kTile, see.last), a.d, lane) ||
           any_not_finite<T>(t, b, kh, max(low, see.first_end), min(see.last, high), a.d, lane) ||
           any_not_finite<T>(t, b, kh, max(max(0, p + 1), low), high, a.d, lane);
}

// Of key j in the tile of keys from k0: the queries and their gradients.
template <class T>
__device__ __noinline__ bool masked_queries_not_finite(const AttentionArgs &a, int b, int kh, int k0, int j) {
    const int lane = threadIdx.x % 32, shift = a.sk - a.sq;
    const QueryTiles tiles = query_tiles(a, k0);
    const int low = tiles.low * kTile, high = min(tiles.high * kTile, a.sq);
    const int i0 = max(0, j - shift), i1 = max(i0, last_position(a, j) - shift + 1);
    for (int h = kh * a.group; h < (kh + 1) * a.group; ++h)
        if (any_not_finite<T>(a.q, b, h, low, min(i0, high), a.d, lane) || any_not_finite<T>(a.d_o, b, h, low, min(i0, high), a.d, lane) ||
            any_not_finite<T>(a.q, b, h, max(i1, low), high, a.d, lane) || any_not_finite<T>(a.d_o, b, h, max(i1, low), high, a.d, lane))
            return true;
    return false;
}

// Whether dS of query i, of the tile from r0, can have been past fp16.
template <class T> __device__ __noinline__ bool dq_past_half(const AttentionArgs &a, int b, int h, int r0, int i) {
    const int lane = threadIdx.x % 32;
    const KeyTiles tiles = key_tiles(a, r0);
    const float *tops = a.v_peak + (int64_t(b) * a.hkv + h / a.group) * ((a.sk + kTile - 1) / kTile);
    float v = 0.f, sum = 0.f;
    for (int j = lane; j < tiles.first; j += 32) v = fmaxf(v, tops[j]);
    for (int j = tiles.low + lane; j < tiles.high; j += 32) v = fmaxf(v, tops[j]);
    const T *row = row_of<const T>(a.d_o, b, i, h);
    for (int e = lane; e < a.d; e += 32) {
        const float x = fabsf(Elem<T>::to_float(row[e]));
        sum += x < INFINITY ? x : 0.f;
    }
    const int64_t at = (int64_t(b) * a.hq + h) * a.sq_pad + i;
    const float d = fabsf(a.stats[at].y);
    return d < INFINITY && past_half(a.unit[at], warp_add(sum), warp_max(v), d);
}

template <class T>
__device__ __forceinline__ void mend_dq_row(const AttentionArgs &a, int b, int h, int r0, int i) {
    bool past = false;
    if constexpr (kUnits<T>) past = dq_past_half<T>(a, b, h, r0, i);
    if (past || masked_keys_not_finite<T>(a, a.k, b, h / a.group, r0, i + a.sk - a.sq)) dq_row<T>(a, b, h, i);
}
// `past`: something can have been past the type's range.
template <class T>
__device__ __forceinline__ void mend_dkv_row(const AttentionArgs &a, int b, int kh, int k0, int j, bool past) {
    if (past || masked_queries_not_finite<T>(a, b, kh, k0, j)) dkv_row<T>(a, b, kh, j);
}

}  // namespace basp_fp8
