// fp8_common.cuh -- what the 8-bit operators share: element types, the scale
// rule, e4m3 conversion, and launch helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <type_traits>

#include "basp_fp8.h"

namespace basp_fp8 {

constexpr int kBlock = BASP_FP8_BLOCK;

// ---- element types --------------------------------------------------------

template <class T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float to_float(float x) { return x; }
    static __device__ __forceinline__ float from_float(float x) { return x; }
};
template <> struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
    static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
};

template <class T> struct alignas(4 * sizeof(T)) Vec4 { T v[4]; };

// 16 bytes of a row as they lie in memory: eight 16-bit values or four of 32
// bits.  max_abs is elementwise: the larger magnitude, a NaN not counted, in
// one instruction for two 16-bit values; the result's signs mean nothing
// (`magnitude` takes them off).
template <class T> struct Pack;
template <> struct Pack<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 x, float (&v)[4]) {
        v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t x) {
        return __float_as_uint(fmaxf(fabsf(__uint_as_float(m)), fabsf(__uint_as_float(x))));
    }
    static __device__ __forceinline__ uint32_t magnitude(uint32_t x) { return x & 0x7fffffffu; }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 x, float (&v)[8]) {
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t x) {
        uint32_t r;
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
        return r;
    }
    static __device__ __forceinline__ uint32_t magnitude(uint32_t x) { return x & 0x7fff7fffu; }
    // the float bits of the low and the high value
    static __device__ __forceinline__ uint32_t low(uint32_t x) { return x << 16; }
    static __device__ __forceinline__ uint32_t high(uint32_t x) { return x & 0xffff0000u; }
};
template <> struct Pack<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 x, float (&v)[8]) {
        const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    static __device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t x) {
        uint32_t r;
        asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x));
        return r;
    }
    static __device__ __forceinline__ uint32_t magnitude(uint32_t x) { return x & 0x7fff7fffu; }
    static __device__ __forceinline__ uint32_t low(uint32_t x) {
        return __float_as_uint(__half2float(__ushort_as_half(uint16_t(x))));
    }
    static __device__ __forceinline__ uint32_t high(uint32_t x) {
        return __float_as_uint(__half2float(__ushort_as_half(uint16_t(x >> 16))));
    }
};

// How a warp's lanes touch a 128-block, four values each.
//   kVector: columns 4*lane .. 4*lane+3 in one access (rows aligned to four
//            elements, and their number a multiple of four)
//   kStrided: columns lane, lane+32, lane+64, lane+96, so that a warp's
//            accesses still fall next to each other, whatever the alignment
//   kWhole:  as kStrided for a block that ends inside its row: no checks, so
//            that the loads of several blocks go out together
enum : int { kStrided = 0, kVector = 1, kWhole = 2 };
template <int HOW> using How = std::integral_constant<int, HOW>;

// `row` points to the block's first element; `left` columns of the block
// exist.  Values past the end read as zero.
template <class T, int HOW>
__device__ __forceinline__ void load4(const T *row, int lane, int left, float (&v)[4]) {
    if constexpr (HOW == kVector) {
        if (4 * lane < left) {            // left % 4 == 0 whenever kVector
            const Vec4<T> x = *reinterpret_cast<const Vec4<T> *>(row + 4 * lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = Elem<T>::to_float(x.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = HOW == kWhole || lane + 32 * j < left ? Elem<T>::to_float(row[lane + 32 * j]) : 0.f;
    }
}

// ---- loads ahead of their use -----------------------------------------------

// A thread copies the 16 bytes that it will read itself into shared memory
// (cp.async: no register holds them on the way, and no barrier is needed to
// read one's own copies).  `have` false: zeros, and nothing is read.
__device__ __forceinline__ void copy16_async(uint4 *dst, const void *src, bool have) {
    const uint32_t to = uint32_t(__cvta_generic_to_shared(dst));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(have ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest N groups of this thread have arrived
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <class T, int HOW>
__device__ __forceinline__ void store4(T *row, int lane, int left, const float (&v)[4]) {
    if constexpr (HOW == kVector) {
        if (4 * lane < left) {
            Vec4<T> x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x.v[j] = Elem<T>::from_float(v[j]);
            *reinterpret_cast<Vec4<T> *>(row + 4 * lane) = x;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (HOW == kWhole || lane + 32 * j < left) row[lane + 32 * j] = Elem<T>::from_float(v[j]);
    }
}

// ---- the scale rule -------------------------------------------------------

constexpr uint32_t kInfBits = 0x7f800000u;

// The largest magnitude's bits, NaN aside: magnitudes order as their bits do,
// so maxima of several lanes are integer maxima.  Infinities count; a block
// where this says kInfBits takes the forms below that look at each value.
__device__ __forceinline__ uint32_t max_bits4(const float (&v)[4]) {
    return __float_as_uint(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
}

// The magnitude's bits where x is finite, else 0.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < kInfBits ? b : 0u;
}
__device__ __forceinline__ uint32_t max_finite_bits4(const float (&v)[4]) {
    return max(max(finite_bits(v[0]), finite_bits(v[1])), max(finite_bits(v[2]), finite_bits(v[3])));
}

// The biased exponent e + 127 of the least scale 2^e with amax <= 448 * 2^e:
// with amax = m * 2^x, 1 <= m < 2, that is e = x - 8 for m <= 1.75 (448 is
// 1.75 * 2^8) and x - 7 above; adding 2^21 - 1 to the bits carries into the
// exponent exactly for m > 1.75.  Subnormal amax reads as x = -127, and e
// stops at -127; a block of zeros has e = 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits == 0u) return 127u;
    const int e = int((amax_bits + 0x1fffffu) >> 23) - 8;
    return e > 0 ? uint32_t(e) : 0u;
}

// 2^-e for a scale byte e + 127 in [0, 247] (amax below 2^128 keeps e <= 120):
// biased exponent 254 - byte, always a normal number.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}

// Four values times the inverse scale, rounded to nearest even: e4m3 bytes,
// the first in the low byte.  NaN gives NaN; an infinity would saturate.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d, float inv) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b * inv), "f"(a * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d * inv), "f"(c * inv));
    return uint32_t(lo) | (uint32_t(hi) << 16);
}
__device__ __forceinline__ uint32_t to_e4m3x4(const float (&v)[4], float inv) {
    return to_e4m3x4(v[0], v[1], v[2], v[3], inv);
}
// the bytes of N = 4 or 8 values to memory
template <int N> __device__ __forceinline__ void store_e4m3(uint8_t *out, const float (&v)[N], float inv) {
    const uint32_t lo = to_e4m3x4(v[0], v[1], v[2], v[3], inv);
    if constexpr (N == 8)
        *reinterpret_cast<uint2 *>(out) = make_uint2(lo, to_e4m3x4(v[4], v[5], v[6], v[7], inv));
    else
        *reinterpret_cast<uint32_t *>(out) = lo;
}

// Infinities as NaN, which e4m3 can hold; other values as they are.
template <int N> __device__ __forceinline__ void infinite_to_nan(float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j)
        if ((__float_as_uint(v[j]) & 0x7fffffffu) == kInfBits) v[j] = __uint_as_float(0x7fffffffu);
}

// The scale byte of a 1 x 128 block that a warp holds; infinities become NaN.
__device__ __forceinline__ uint32_t row_scale(float (&v)[4]) {
    uint32_t m = __reduce_max_sync(0xffffffffu, max_bits4(v));
    if (m >= kInfBits) {
        m = __reduce_max_sync(0xffffffffu, max_finite_bits4(v));
        infinite_to_nan(v);
    }
    return scale_byte(m);
}

template <int HOW>
__device__ __forceinline__ void store4_e4m3(uint8_t *row, int lane, int left, uint32_t q) {
    if constexpr (HOW == kVector) {
        if (4 * lane < left) *reinterpret_cast<uint32_t *>(row + 4 * lane) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (HOW == kWhole || lane + 32 * j < left) row[lane + 32 * j] = uint8_t(q >> (8 * j));
    }
}

// ---- launch ---------------------------------------------------------------

// Wait for the previous kernel on the stream (nothing is read or written
// before), then let the next one be scheduled; it waits the same way.
__device__ __forceinline__ void grid_dependency() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launch with programmatic dependent launch, and a cluster along x if > 1.
template <class... P, class... A>
basp_status launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster,
                   cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, P(args)...) != cudaSuccess) {
        cudaGetLastError();               // clear the error this launch set
        return BASP_ERR_CUDA;
    }
    return BASP_OK;
}

// An NVTX range named after the entry point (a no-op without a tool).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

// SMs of a GB300, for sizes that a host without one has to know too (workspaces).
constexpr int kSms = 152;

// SMs of the current device (152 on GB300); 1 if it cannot be read.
int sm_count();

// Lets KERNEL have up to MOST bytes of dynamic shared memory.  The limit belongs
// to the function, for all host threads: each call sets the same one, whatever
// its own launch needs, so none lowers it between another's setting and launch.
template <auto KERNEL, size_t MOST> bool allow_shared_memory() {
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, int(MOST)) == cudaSuccess) return true;
    cudaGetLastError();
    return false;
}

// CTAs of `kernel` that fit on the current device at once.
template <class K>
int64_t resident_ctas(K kernel, int threads, size_t smem) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess) {
        cudaGetLastError();
        per_sm = 1;
    }
    return int64_t(sm_count()) * (per_sm > 0 ? per_sm : 1);
}

// ---- argument checks (host) -----------------------------------------------

inline int64_t elem_size(basp_dtype t) {
    switch (t) {
        case BASP_DTYPE_BF16: case BASP_DTYPE_FP16: return 2;
        case BASP_DTYPE_FP32: return 4;
        default: return 0;                // not an element type of these calls
    }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxSide = (int64_t(1) << 31) - 1;

// The bytes [lo, hi) a buffer spans.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool touches(const Span &o) const { return lo < o.hi && o.lo < hi; }
};

// Collects a call's buffers and its first error; status() also tells whether
// an output overlaps another buffer.
class Args {
  public:
    // a row-major matrix; ok to be NULL unless `need`
    void matrix(const void *p, int64_t rows, int64_t cols, int64_t stride, int64_t esz, bool out,
                bool need = true) {
        if (p == nullptr) {
            if (need && rows > 0 && cols > 0) fail(BASP_ERR_INVALID_ARG);
            return;
        }
        if (rows <= 0 || cols <= 0) return;
        if (rows > 1 && stride < cols) return fail(BASP_ERR_INVALID_ARG);
        if (stride < 0) return fail(BASP_ERR_INVALID_ARG);
        if (uintptr_t(p) % uintptr_t(esz)) return fail(BASP_ERR_ALIGNMENT);
        int64_t last;
        if (__builtin_mul_overflow(rows - 1, stride, &last) || last > (int64_t(1) << 58))
            return fail(BASP_ERR_TOO_LARGE);
        add(p, (last + cols) * esz, out);
    }
    void fp8(const basp_fp8_matrix *m, int64_t rows, int64_t cols, bool out) {
        if (m->rows != rows || m->cols != cols || (m->block_rows != 1 && m->block_rows != kBlock))
            return fail(BASP_ERR_INVALID_ARG);
        if (rows == 0 || cols == 0) return;
        if (m->data == nullptr || m->scales == nullptr) return fail(BASP_ERR_INVALID_ARG);
        if (m->pitch < cols || m->scale_pitch < ceil_div(cols, kBlock))
            return fail(BASP_ERR_INVALID_ARG);
        if (m->pitch % 16 || uintptr_t(m->data) % 16 || m->scale_pitch % 4 || uintptr_t(m->scales) % 4)
            return fail(BASP_ERR_ALIGNMENT);
        matrix(m->data, rows, cols, m->pitch, 1, out);
        matrix(m->scales, ceil_div(rows, m->block_rows), ceil_div(cols, kBlock), m->scale_pitch, 1, out);
    }
    // an output that may be the very buffer of an input: same start and end
    void allow_same(const void *out, const void *in) {
        if (out != nullptr && out == in) same_[nsame_++] = uintptr_t(out);
    }
    void fail(basp_status s) { if (status_ == BASP_OK) status_ = s; }
    basp_status status() const {
        if (status_ != BASP_OK) return status_;
        for (int i = 0; i < n_; ++i)
            for (int j = 0; j < n_; ++j) {
                if (i == j || !out_[i] || !span_[i].touches(span_[j])) continue;
                bool ok = false;
                for (int k = 0; k < nsame_; ++k)
                    ok |= !out_[j] && span_[i].lo == same_[k] && span_[j].lo == same_[k] &&
                          span_[i].hi == span_[j].hi;
                if (!ok) return BASP_ERR_ALIASING;
            }
        return BASP_OK;
    }

  private:
    void add(const void *p, int64_t bytes, bool out) {
        span_[n_].lo = uintptr_t(p);
        span_[n_].hi = uintptr_t(p) + uintptr_t(bytes);
        out_[n_++] = out;
    }
    basp_status status_ = BASP_OK;
    Span span_[12];
    bool out_[12] = {};
    int n_ = 0;
    uintptr_t same_[4] = {};
    int nsame_ = 0;
};

inline bool sides_ok(int64_t rows, int64_t cols, basp_status *st) {
    if (rows < 0 || cols < 0) { *st = BASP_ERR_INVALID_ARG; return false; }
    if (rows > kMaxSide || cols > kMaxSide) { *st = BASP_ERR_TOO_LARGE; return false; }
    return true;
}

// Whether rows of `stride` elements of `esz` bytes at p (NULL counts) and
// `cols` allow accesses of 16 bytes.
inline bool vec16_ok(const void *p, int64_t stride, int64_t cols, int64_t esz) {
    return p == nullptr || (uintptr_t(p) % 16 == 0 && stride * esz % 16 == 0 && cols * esz % 16 == 0);
}

// Whether they allow accesses of four elements.
inline bool vec4_ok(const void *p, int64_t stride, int64_t cols, int64_t esz) {
    return p == nullptr || (uintptr_t(p) % uintptr_t(4 * esz) == 0 && stride % 4 == 0 && cols % 4 == 0);
}

}  // namespace basp_fp8
