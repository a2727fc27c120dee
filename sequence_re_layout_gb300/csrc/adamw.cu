// adamw.cu -- one step of Adam with decoupled weight decay over many tensors
// (basp_adamw).
//
// The bound is memory: with 32-bit weights and gradients 28 bytes an element with
// 32-bit states, 16 with 8-bit ones.  One launch takes a table of tensors as its
// parameter (up to 32 KB, copied with the launch, so there is nothing to keep or to
// upload) and a grid of chunks; a CTA finds its chunk's tensor by bisection.
//
// 50 million fp32 values: 204 us, at a copy's rate (some of it stays in L2).  Four such with
// 8-bit states: 560 us, 0.86 of a copy's rate; issue slots bound it (86 % of them), 46 us of it
// the root to its last bit.
//
// 8-bit states have a scale for each 128 elements, which one warp holds, four a
// lane, so the largest magnitude is one warp reduction and nothing is read twice.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "basp_optim.h"
#include "fp8_common.cuh"

namespace basp_fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 128 * (kThreads / 32) * 16;       // elements of a CTA

struct Entry {
    void *p;
    const void *g;
    void *m, *v, *ms, *vs;
    const int32_t *step_at;                          // its step's number, or NULL: Options::step
    int64_t n;
    uint32_t number;                                 // for the random bits
    int32_t chunk0;                                  // its first chunk in the launch
    uint8_t type, grad_type, vec, pad[5];
};
static_assert(sizeof(Entry) == 80, "table");

struct Options {
    float beta1, beta2, one_beta1, one_beta2, eps, decay, lr;   // decay: 1 - lr * weight_decay
    float c1, c2;                                    // lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
    float log_beta1, log_beta2;                      // for a t that is known on the GPU only
    uint32_t step, seed;
};

template <int CAP> struct Table {
    Options o;
    int32_t count, pad;                              // entries
    Entry e[CAP];
};

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

// |y| <= 448 to the e4m3 grid, up with probability of the fraction: the 16 bits r
// (and a half, `r` is 16 times that: 16 r + 8) are added below the last of the three
// mantissa bits, which does not reach the sign.
__device__ __forceinline__ float round_normal(float y, uint32_t r) {
    return __uint_as_float((__float_as_uint(y) + r) & 0xfff00000u);
}
// The same for any y: values below 2^-6, whose steps are 2^-9, get there by an addition of
// 2^-6, exact to 2^-29; a NaN stays.
__device__ __forceinline__ float round_any(float y, uint32_t r) {
    const float a = fabsf(y);
    if (!(a <= 448.f)) return y;
    const bool small = a < 0x1p-6f;
    const float t = round_normal(small ? a + 0x1p-6f : a, r);
    return copysignf(small ? t - 0x1p-6f : t, y);
}

// The scale byte of a block from its largest magnitude's bits, or where those say that
// there are infinities or NaN, of what is finite; infinities become NaN.
__device__ __forceinline__ uint32_t state_scale(uint32_t top, float (&v)[4]) {
    if (top >= kInfBits) {
        top = __reduce_max_sync(0xffffffffu, max_finite_bits4(v));
        infinite_to_nan(v);
    }
    return scale_byte(top);
}

__device__ __forceinline__ float scale_of(uint32_t byte) {           // 2^(byte - 127)
    return byte != 0 ? __uint_as_float(byte << 23) : 0x1p-127f;
}
// e4m3 -> float, by way of fp16, which holds every e4m3 value
__device__ __forceinline__ void from_e4m3x4(uint32_t q, float (&v)[4]) {
    uint32_t lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(q)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(q >> 16)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// A quotient to two units in the last place, of a y from 2^-126 to 2^126.
__device__ __forceinline__ float over(float x, float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return x * r;
}

// What a step does to one element; m and v become m' and v', `root` the root of v'.
__device__ __forceinline__ float step_of(const Options &o, float c1, float c2, float p, float g, float &m, float &v,
                                         float &root) {
    // The states' operations are rounded one by one, as 32-bit arithmetic has them and not
    // fused: a state is then the same, down to which way it is rounded at random, as that of
    // any other program that follows the formula in 32 bits.
    m = __fadd_rn(__fmul_rn(o.beta1, m), __fmul_rn(o.one_beta1, g));
    v = __fadd_rn(__fmul_rn(o.beta2, v), __fmul_rn(o.one_beta2, __fmul_rn(g, g)));
    root = __fsqrt_rn(v);
    return fmaf(p, o.decay, -c1 * over(m, fmaf(root, c2, o.eps)));
}

// Four elements of a 128-block (load4 of fp8_common.cuh), or their state bytes.
template <int HOW> __device__ __forceinline__ uint32_t load4_bytes(const uint8_t *row, int lane, int left) {
    if constexpr (HOW == kVector) return 4 * lane < left ? *reinterpret_cast<const uint32_t *>(row + 4 * lane) : 0u;
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < left) q |= uint32_t(row[lane + 32 * j]) << (8 * j);
    return q;
}

// One block of 128 with 8-bit states: p, g and the state bytes (four a lane) as they were,
// p and the state bytes as they will be, and the scale bytes.  `at`: the block's first
// element's place in its tensor.
template <int HOW>
__device__ __forceinline__ void step_block(const Options &o, float c1, float c2, uint32_t key, uint32_t at, float (&p)[4],
                                           const float (&g)[4], uint32_t &qm, uint32_t &qv, uint32_t &em, uint32_t &ev) {
    const int lane = threadIdx.x % 32;
    float m[4], v[4], root[4];
    from_e4m3x4(qm, m);
    from_e4m3x4(qv, v);
    const float sm = scale_of(em), sv = scale_of(ev);
    uint32_t bits[4], tm = 0, tv = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        m[j] *= sm;
        v[j] *= sv;
        v[j] *= v[j];
        p[j] = step_of(o, c1, c2, p[j], g[j], m[j], v[j], root[j]);
        bits[j] = __float_as_uint(m[j]) & 0x7fffffffu;
        tm = max(tm, bits[j]);
        tv = max(tv, __float_as_uint(root[j]) & 0x7fffffffu);
    }
    tm = __reduce_max_sync(0xffffffffu, tm);
    tv = __reduce_max_sync(0xffffffffu, tv);
    em = state_scale(tm, m);                              // infinities are NaN now
    ev = state_scale(tv, root);
    const float im = inverse_scale(em), iv = inverse_scale(ev);
    float a[4], b[4];
    uint32_t r[4];
    bool plain = max(tm, tv) < kInfBits;                  // and no value but 0 below the 8 bits' normal range
    const uint32_t lm = __float_as_uint(0x1p-6f * scale_of(em)) - 1, lv = __float_as_uint(0x1p-6f * scale_of(ev)) - 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r[j] = mix((at + uint32_t(HOW == kVector ? 4 * lane + j : lane + 32 * j)) * 0x9E3779B9u + key);
        a[j] = m[j] * im;
        b[j] = root[j] * iv;
        plain = plain && bits[j] - 1 >= lm && __float_as_uint(root[j]) - 1 >= lv;
    }
    if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = round_normal(a[j], (r[j] << 4 & 0xffff0u) | 8u);
            b[j] = round_normal(b[j], (r[j] >> 12 & 0xffff0u) | 8u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = round_any(a[j], (r[j] << 4 & 0xffff0u) | 8u);
            const float y = b[j];
            b[j] = round_any(y, (r[j] >> 12 & 0xffff0u) | 8u);
            if (y > 0.f) b[j] = fmaxf(b[j], 0x1p-9f);
        }
    }
    qm = to_e4m3x4(a, 1.f);
    qv = to_e4m3x4(b, 1.f);
}

// A chunk with 32-bit states.
template <class P, class G, int HOW>
__device__ __forceinline__ void do_chunk32(const Entry &e, const Options &o, float c1, float c2, int64_t begin) {
    constexpr int kBlocksEach = 4;                        // blocks of 128 that a warp has on their way at once
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = kThreads / 32;
    const int64_t end = min(e.n, begin + kChunk);
    for (int64_t b0 = begin + int64_t(warp) * kBlocksEach * kBlock; b0 < end; b0 += int64_t(warps) * kBlocksEach * kBlock) {
        float p[kBlocksEach][4], g[kBlocksEach][4], m[kBlocksEach][4], v[kBlocksEach][4], root;
#pragma unroll
        for (int i = 0; i < kBlocksEach; ++i) {
            const int64_t at = b0 + i * kBlock;
            const int left = int(max(int64_t(0), min(end - at, int64_t(kBlock))));
            load4<P, HOW>(static_cast<const P *>(e.p) + at, lane, left, p[i]);
            load4<G, HOW>(static_cast<const G *>(e.g) + at, lane, left, g[i]);
            load4<float, HOW>(static_cast<const float *>(e.m) + at, lane, left, m[i]);
            load4<float, HOW>(static_cast<const float *>(e.v) + at, lane, left, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kBlocksEach; ++i) {
            const int64_t at = b0 + i * kBlock;
            const int left = int(max(int64_t(0), min(end - at, int64_t(kBlock))));
#pragma unroll
            for (int j = 0; j < 4; ++j) p[i][j] = step_of(o, c1, c2, p[i][j], g[i][j], m[i][j], v[i][j], root);
            store4<P, HOW>(static_cast<P *>(e.p) + at, lane, left, p[i]);
            store4<float, HOW>(static_cast<float *>(e.m) + at, lane, left, m[i]);
            store4<float, HOW>(static_cast<float *>(e.v) + at, lane, left, v[i]);
        }
    }
}

// A chunk with 8-bit states, whose warps have 16 neighbouring blocks each: the scale
// bytes of those are one load, and one store at the end.
constexpr int kRun = kChunk / kBlock / (kThreads / 32);
static_assert(kRun == 16, "a lane for each scale of a run, of m and of v");

// The buffers allow four elements at a time: each lane copies what it will read itself
// to shared memory, kStages - 1 blocks ahead.  What bounds this kernel otherwise is the
// number of bytes in flight: 1165 us for four layers of 50 million elements, not 560, with
// the loads of two blocks in registers.
constexpr int kStages = 4, kStageBytes = 32 * (16 + 16 + 4 + 4);

template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool have) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                     ::"r"(dst), "l"(src), "n"(BYTES), "r"(have ? BYTES : 0) : "memory");
}

template <class P, class G, int HOW>
__device__ __forceinline__ void do_chunk8(const Entry &e, const Options &o, float c1, float c2, uint32_t key, int64_t begin,
                                          uint8_t *ring) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t first = begin + int64_t(warp) * kRun * kBlock;
    if (first >= e.n) return;
    const int blocks = int(min(int64_t(kRun), (e.n - first + kBlock - 1) / kBlock));
    uint8_t *const scales = static_cast<uint8_t *>(lane < kRun ? e.ms : e.vs) + first / kBlock + lane % kRun;
    const uint32_t old = lane % kRun < blocks ? *scales : 0u;
    uint32_t made = 0;
    uint8_t *mine = ring + warp * (kStages * kStageBytes);
    const P *ep = static_cast<const P *>(e.p) + first;
    const G *eg = static_cast<const G *>(e.g) + first;
    const uint8_t *m8 = static_cast<const uint8_t *>(e.m) + first, *v8 = static_cast<const uint8_t *>(e.v) + first;
    auto left_of = [&](int i) { return int(min(e.n - first - int64_t(i) * kBlock, int64_t(kBlock))); };
    auto fetch = [&](int i) {
        if constexpr (HOW == kVector) {
            if (i < blocks) {
                const uint32_t to = uint32_t(__cvta_generic_to_shared(mine + (i % kStages) * kStageBytes));
                const bool have = 4 * lane < left_of(i);
                const int at = have ? i * kBlock + 4 * lane : 0;
                copy_async<4 * sizeof(P)>(to + lane * 16, ep + at, have);
                copy_async<4 * sizeof(G)>(to + 512 + lane * 16, eg + at, have);
                copy_async<4>(to + 1024 + lane * 4, m8 + at, have);
                copy_async<4>(to + 1152 + lane * 4, v8 + at, have);
            }
            copy_commit();                                // an empty group past the end keeps the count
        }
    };
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
#pragma unroll 1
    for (int i = 0; i < blocks; ++i) {
        const int left = left_of(i);
        float p[4], g[4];
        uint32_t qm, qv;
        fetch(i + kStages - 1);
        if constexpr (HOW == kVector) {
            copy_wait<kStages - 1>();
            const uint8_t *from = mine + (i % kStages) * kStageBytes;
            load4<P, kVector>(reinterpret_cast<const P *>(from + lane * 16), 0, 4, p);
            load4<G, kVector>(reinterpret_cast<const G *>(from + 512 + lane * 16), 0, 4, g);
            qm = *reinterpret_cast<const uint32_t *>(from + 1024 + lane * 4);
            qv = *reinterpret_cast<const uint32_t *>(from + 1152 + lane * 4);
        } else {
            load4<P, HOW>(ep + i * kBlock, lane, left, p);
            load4<G, HOW>(eg + i * kBlock, lane, left, g);
            qm = load4_bytes<HOW>(m8 + i * kBlock, lane, left);
            qv = load4_bytes<HOW>(v8 + i * kBlock, lane, left);
        }
        uint32_t em = __shfl_sync(0xffffffffu, old, i), ev = __shfl_sync(0xffffffffu, old, i + kRun);
        step_block<HOW>(o, c1, c2, key, uint32_t(first + i * kBlock), p, g, qm, qv, em, ev);
        store4<P, HOW>(static_cast<P *>(e.p) + first + i * kBlock, lane, left, p);
        store4_e4m3<HOW>(static_cast<uint8_t *>(e.m) + first + i * kBlock, lane, left, qm);
        store4_e4m3<HOW>(static_cast<uint8_t *>(e.v) + first + i * kBlock, lane, left, qv);
        if (lane % kRun == i) made = lane < kRun ? em : ev;
    }
    if (lane % kRun < blocks) *scales = uint8_t(made);
}

template <int CAP, bool EIGHT>
__global__ void __launch_bounds__(kThreads, EIGHT ? 4 : 2) adamw_kernel(const __grid_constant__ Table<CAP> t) {
    __shared__ __align__(16) uint8_t ring[EIGHT ? (kThreads / 32) * kStages * kStageBytes : 16];
    grid_dependency();
    int lo = 0, hi = t.count;                        // e[lo].chunk0 <= chunk < e[hi].chunk0
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.e[mid].chunk0 <= int(blockIdx.x)) lo = mid;
        else hi = mid;
    }
    const Entry &e = t.e[lo];
    const int64_t begin = int64_t(int(blockIdx.x) - e.chunk0) * kChunk;
    float c1 = t.o.c1, c2 = t.o.c2;
    uint32_t step = t.o.step;
    if (e.step_at != nullptr) {
        const int s = max(1, *e.step_at);
        step = uint32_t(s);
        c1 = t.o.lr / -expm1f(float(s) * t.o.log_beta1);
        c2 = rsqrtf(-expm1f(float(s) * t.o.log_beta2));
    }
    const uint32_t key = EIGHT ? mix(mix(mix(t.o.seed) ^ step) ^ e.number) : 0u;
    auto go = [&](auto pe, auto ge) {
        using P = decltype(pe);
        using G = decltype(ge);
        if constexpr (EIGHT) {
            if (e.vec) do_chunk8<P, G, kVector>(e, t.o, c1, c2, key, begin, ring);
            else do_chunk8<P, G, kStrided>(e, t.o, c1, c2, key, begin, ring);
        } else {
            if (e.vec) do_chunk32<P, G, kVector>(e, t.o, c1, c2, begin);
            else do_chunk32<P, G, kStrided>(e, t.o, c1, c2, begin);
        }
    };
    if (e.type == BASP_DTYPE_FP32) return go(float(), float());
    if (e.type == BASP_DTYPE_BF16)
        return e.grad_type == BASP_DTYPE_FP32 ? go(__nv_bfloat16(), float()) : go(__nv_bfloat16(), __nv_bfloat16());
    return e.grad_type == BASP_DTYPE_FP32 ? go(__half(), float()) : go(__half(), __half());
}

int64_t chunks_of(int64_t n) { return ceil_div(n, kChunk); }

// One launch of entries [i0, i1) of the caller's list.
template <int CAP>
basp_status launch_adamw(const basp_adamw_tensor *list, const int32_t *const *steps_at, const uint32_t *numbers, int64_t i0,
                         int64_t i1, bool eight, const Options &o, const int32_t *step_at, int64_t *next, cudaStream_t stream) {
    Table<CAP> t;
    t.o = o;
    t.count = 0;
    t.pad = 0;
    int64_t chunks = 0, i = i0;
    for (; i < i1 && t.count < CAP; ++i) {
        const basp_adamw_tensor &x = list[i];
        const int64_t c = chunks_of(x.n);
        if (chunks + c > kMaxSide) break;            // the next launch
        Entry &e = t.e[t.count++];
        e.p = x.p; e.g = x.g; e.m = x.m; e.v = x.v; e.ms = x.m_scales; e.vs = x.v_scales;
        e.step_at = steps_at != nullptr ? steps_at[i] : step_at;
        e.n = x.n;
        e.number = numbers != nullptr ? numbers[i] : uint32_t(i);
        e.chunk0 = int32_t(chunks);
        e.type = uint8_t(x.dtype);
        e.grad_type = uint8_t(x.grad_dtype);
        // the last block's four elements of a lane may be past the end
        const int64_t state = eight ? 1 : 4;
        e.vec = x.n % 4 == 0 && vec4_ok(x.p, 0, x.n, elem_size(x.dtype)) && vec4_ok(x.g, 0, x.n, elem_size(x.grad_dtype)) &&
                vec4_ok(x.m, 0, x.n, state) && vec4_ok(x.v, 0, x.n, state);
        std::fill(e.pad, e.pad + sizeof(e.pad), uint8_t(0));
        chunks += c;
    }
    *next = i;
    if (chunks == 0) return BASP_OK;
    // launch() of fp8_common.cuh would copy the table twice more
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(chunks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void *args[] = {&t};
    const void *kernel = eight ? reinterpret_cast<const void *>(adamw_kernel<CAP, true>)
                               : reinterpret_cast<const void *>(adamw_kernel<CAP, false>);
    if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
        cudaGetLastError();
        return BASP_ERR_CUDA;
    }
    return BASP_OK;
}

basp_status check_tensor(const basp_adamw_tensor &x, bool eight) {
    const int64_t ps = elem_size(x.dtype), gs = elem_size(x.grad_dtype);
    if (ps == 0 || gs == 0 || (x.grad_dtype != x.dtype && x.grad_dtype != BASP_DTYPE_FP32) || x.n < 0)
        return BASP_ERR_INVALID_ARG;
    if (x.n == 0) return BASP_OK;
    if ((x.m_scales != nullptr) != eight || (x.v_scales != nullptr) != eight) return BASP_ERR_INVALID_ARG;
    if (chunks_of(x.n) > kMaxSide) return BASP_ERR_TOO_LARGE;
    const int64_t ss = eight ? 1 : 4, scales = eight ? ceil_div(x.n, kBlock) : 0;
    if (x.n > (int64_t(1) << 56)) return BASP_ERR_TOO_LARGE;
    // p, g, m, v and the scales: there, aligned, and apart
    const struct { const void *p; int64_t bytes, size; } s[6] = {
        {x.p, x.n * ps, ps}, {x.g, x.n * gs, gs}, {x.m, x.n * ss, ss}, {x.v, x.n * ss, ss},
        {x.m_scales, scales, 1}, {x.v_scales, scales, 1}};
    for (int i = 0; i < (eight ? 6 : 4); ++i) {
        const uintptr_t at = uintptr_t(s[i].p);
        if (at == 0) return BASP_ERR_INVALID_ARG;
        if (at % uintptr_t(s[i].size)) return BASP_ERR_ALIGNMENT;
        for (int j = 0; j < i; ++j) {
            const uintptr_t other = uintptr_t(s[j].p);
            if (at < other + uintptr_t(s[j].bytes) && other < at + uintptr_t(s[i].bytes)) return BASP_ERR_ALIASING;
        }
    }
    return BASP_OK;
}

// No parameter comes twice: two CTAs would update it at a time.
basp_status check_apart(const basp_adamw_tensor *list, int64_t count) {
    struct Span {
        uintptr_t begin, end;
        bool operator<(const Span &o) const { return begin < o.begin; }
    };
    constexpr int64_t kFew = 512;
    Span few[kFew];
    std::unique_ptr<Span[]> many(count > kFew ? new (std::nothrow) Span[size_t(count)] : nullptr);
    if (count > kFew && many == nullptr) return BASP_ERR_TOO_LARGE;
    Span *s = count > kFew ? many.get() : few;
    int64_t n = 0;
    bool rising = true;                              // as tensors from one allocator often are
    for (int64_t i = 0; i < count; ++i) {
        if (list[i].n == 0) continue;
        const uintptr_t at = uintptr_t(list[i].p);
        rising = rising && (n == 0 || s[n - 1].begin <= at);
        s[n++] = {at, at + uintptr_t(list[i].n * elem_size(list[i].dtype))};
    }
    if (!rising) std::sort(s, s + n);
    for (int64_t i = 1; i < n; ++i)
        if (s[i].begin < s[i - 1].end) return BASP_ERR_ALIASING;
    return BASP_OK;
}

basp_status adamw(const basp_adamw_tensor *tensors, const int32_t *const *steps_at, const uint32_t *numbers, int64_t count,
                  const basp_adamw_options *options, cudaStream_t stream) {
    if (count < 0 || options == nullptr || (tensors == nullptr && count > 0)) return BASP_ERR_INVALID_ARG;
    const basp_adamw_options &p = *options;
    // a comparison that a NaN fails
    if (!(p.lr >= 0 && p.lr < INFINITY && p.beta1 >= 0 && p.beta1 < 1 && p.beta2 >= 0 && p.beta2 < 1 && p.eps >= 0 &&
          p.eps < INFINITY && p.weight_decay >= 0 && p.weight_decay < INFINITY))
        return BASP_ERR_INVALID_ARG;
    const bool counted = steps_at == nullptr && p.step_at == nullptr;      // t is the options' step
    if (counted && (p.step < 1 || p.step > kMaxSide)) return BASP_ERR_INVALID_ARG;
    if (steps_at == nullptr && uintptr_t(p.step_at) % 4) return BASP_ERR_ALIGNMENT;
    if (count > kMaxSide) return BASP_ERR_TOO_LARGE;
    bool eight = false;
    for (int64_t i = 0; i < count; ++i)
        if (tensors[i].n > 0) {
            eight = tensors[i].m_scales != nullptr;
            break;
        }
    for (int64_t i = 0; i < count; ++i) {
        const basp_status st = check_tensor(tensors[i], eight);
        if (st != BASP_OK) return st;
        if (steps_at != nullptr && tensors[i].n > 0 && steps_at[i] == nullptr) return BASP_ERR_INVALID_ARG;
        if (steps_at != nullptr && uintptr_t(steps_at[i]) % 4) return BASP_ERR_ALIGNMENT;
    }
    if (const basp_status apart = check_apart(tensors, count); apart != BASP_OK) return apart;

    Options o = {};
    o.beta1 = float(p.beta1); o.beta2 = float(p.beta2);
    o.one_beta1 = float(1 - p.beta1); o.one_beta2 = float(1 - p.beta2);
    o.eps = float(p.eps); o.decay = float(1 - p.lr * p.weight_decay); o.lr = float(p.lr);
    o.seed = p.seed;
    if (counted) {
        o.step = uint32_t(p.step);
        o.c1 = float(p.lr / (1 - std::pow(p.beta1, double(p.step))));
        o.c2 = float(1 / std::sqrt(1 - std::pow(p.beta2, double(p.step))));
    } else {
        o.log_beta1 = float(std::log(p.beta1));      // of 0: minus infinity, and beta^t = 0
        o.log_beta2 = float(std::log(p.beta2));
    }
    // Tables of three sizes: a launch copies all of its parameters.
    basp_status st = BASP_OK;
    for (int64_t i = 0; i < count && st == BASP_OK;) {
        auto go = [&](auto cap) {
            st = launch_adamw<decltype(cap)::value>(tensors, steps_at, numbers, i, count, eight, o, p.step_at, &i, stream);
        };
        if (count - i <= 12) go(std::integral_constant<int, 12>());
        else if (count - i <= 60) go(std::integral_constant<int, 60>());
        else go(std::integral_constant<int, 400>());
    }
    return st;
}

}  // namespace
}  // namespace basp_fp8

extern "C" basp_status basp_adamw(const basp_adamw_tensor *tensors, int64_t count, const basp_adamw_options *options,
                                  cudaStream_t stream) {
    basp_fp8::NvtxRange range("basp_adamw");
    return basp_fp8::adamw(tensors, nullptr, nullptr, count, options, stream);
}

extern "C" basp_status basp_adamw_each(const basp_adamw_tensor *tensors, const int32_t *const *steps_at,
                                       const uint32_t *numbers, int64_t count, const basp_adamw_options *options,
                                       cudaStream_t stream) {
    basp_fp8::NvtxRange range("basp_adamw_each");
    return basp_fp8::adamw(tensors, steps_at, numbers, count, options, stream);
}
