// attention_decode.cu -- one new token of each sequence over a cache.
//
// Memory is the bound: the visible keys and values are read once, 4 d flops for each
// 4 d bytes and query head.  A CTA has one key head of one sequence, the (up to 16) query
// heads that share it, and a chunk of the visible keys; four warps take 16 keys at a time
// in turn, each with its own running maximum and sum, and meet in shared memory at the
// end.  Where there is more than one chunk, a second kernel joins the chunks' parts in
// their order.
//
// Keys and values go from memory to registers, 16 bytes a lane, and straight into
// mma.sync (16 query rows x 8 keys or columns x 16): a tcgen05 product would want 128
// rows.  The sum over a head's values may be taken in any order, so lane t of four
// takes the values 8 t + 32 c .. + 7 of a key for both operands, as they lie; for the
// product with V, lane g of eight takes the columns 8 g + 64 c .. + 7 of its four keys, and
// pairs of keys are put together by byte permutations.
#include <algorithm>

#include "attention.cuh"

namespace basp_fp8 {
namespace {

constexpr int kWarps = 4, kKeys = 16, kRows = 16;

struct DecodeArgs {
    AttentionArgs a;
    const int32_t *lengths;
    float *part;                         // [batch][Hq][chunks][d + 2]: sum, maximum, O
    int chunk, chunks, row_blocks;
};

template <class T> __device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The cache is read once: past L1, and first to go from L2.
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <class T, int HD>
__global__ void __launch_bounds__(kWarps * 32, HD == 64 ? 4 : 3) decode_kernel(const __grid_constant__ DecodeArgs p) {
    constexpr int KC = HD / 32, VC = HD / 64;                 // 16-byte pieces of a key, of a value row, a lane
    __shared__ float so[kWarps][kRows][HD + 4];
    __shared__ float sm[kWarps][kRows], sl[kWarps][kRows];
    const AttentionArgs &a = p.a;
    grid_dependency();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int chunk = blockIdx.x, kh = int(blockIdx.y) / p.row_blocks, block = int(blockIdx.y) % p.row_blocks;
    const int rows = min(kRows, a.group - block * kRows), h0 = kh * a.group + block * kRows;
    for (int b = blockIdx.z; b < a.batch; b += gridDim.z) {
        const int len = max(0, min(a.sk, p.lengths[b]));
        const Sees see = keys_of(a, len - 1);
        // the visible keys in a row: [0, first_end), then [low, len)
        const int seen = see.first_end + len - see.last, skip = see.last - see.first_end;
        const int n0 = chunk * p.chunk, n1 = min(seen, n0 + p.chunk);
        if (n0 >= n1 && !(p.chunks == 1 && len == 0)) continue;

        uint32_t q[HD / 16][4];
        {
            const T *r0 = row_of<const T>(a.q, b, 0, h0 + min(g, rows - 1)), *r1 = row_of<const T>(a.q, b, 0, h0 + min(g + 8, rows - 1));
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const bool in = 8 * t + 32 * c < a.d;
                const uint4 x = in ? *reinterpret_cast<const uint4 *>(r0 + 8 * t + 32 * c) : make_uint4(0, 0, 0, 0);
                const uint4 y = in ? *reinterpret_cast<const uint4 *>(r1 + 8 * t + 32 * c) : make_uint4(0, 0, 0, 0);
                q[2 * c][0] = x.x; q[2 * c][1] = y.x; q[2 * c][2] = x.y; q[2 * c][3] = y.y;
                q[2 * c + 1][0] = x.z; q[2 * c + 1][1] = y.z; q[2 * c + 1][2] = x.w; q[2 * c + 1][3] = y.w;
            }
        }
        const T *kp = row_of<const T>(a.k, b, 0, kh), *vp = row_of<const T>(a.v, b, 0, kh);
        uint4 kr[2][KC], vr[4][VC];
        auto load_k = [&](int n) {                            // key g of each eight
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = n + 8 * x + g;
                const T *r = kp + int64_t(i < see.first_end ? i : i + skip) * a.k.ss;
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    kr[x][c] = i < n1 && 8 * t + 32 * c < a.d ? load_once(r + 8 * t + 32 * c) : make_uint4(0, 0, 0, 0);
            }
        };
        auto load_v = [&](int n) {                            // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = n + 8 * (x / 2) + 2 * t + x % 2;
                const T *r = vp + int64_t(i < see.first_end ? i : i + skip) * a.v.ss;
#pragma unroll
                for (int c = 0; c < VC; ++c)
                    vr[x][c] = i < n1 && 8 * g + 64 * c < a.d ? load_once(r + 8 * g + 64 * c) : make_uint4(0, 0, 0, 0);
            }
        };
        float o[HD / 8][4], top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        const float c = a.scale * kLog2e;
        int n = n0 + warp * kKeys;
        load_k(n);
        load_v(n);
        for (; n < n1; n += kWarps * kKeys) {
            float s[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[x][j] = 0.f;
#pragma unroll
                for (int y = 0; y < KC; ++y) {
                    mma_16x8x16<T>(s[x], q[2 * y], kr[x][y].x, kr[x][y].y);
                    mma_16x8x16<T>(s[x], q[2 * y + 1], kr[x][y].z, kr[x][y].w);
                }
            }
            load_k(n + kWarps * kKeys);
            // rows g and g + 8: columns 2 t, 2 t + 1 of each eight keys
            float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[x][j] = n + 8 * x + 2 * t + j % 2 < n1 ? s[x][j] * c : -INFINITY;
                    high[j / 2] = fmaxf(high[j / 2], s[x][j]);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 1));
                high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 2));
                high[r] = fmaxf(high[r], top[r]);
            }
            // raised where it has grown by more than 8: P stays below 2^8
            if (__any_sync(0xffffffffu, high[0] > top[0] + 8.f || high[1] > top[1] + 8.f)) {
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    f[r] = high[r] == -INFINITY ? 1.f : exp2_fast(top[r] - high[r]);
                    top[r] = high[r];
                    l[r] *= f[r];
                }
#pragma unroll
                for (int i = 0; i < HD / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= f[j / 2];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[x][j] = exp2_fast(s[x][j] - (top[j / 2] == -INFINITY ? 0.f : top[j / 2]));
                    l[j / 2] += s[x][j];
                }
            const uint32_t w[4] = {pack_pair<T>(s[0][0], s[0][1]), pack_pair<T>(s[0][2], s[0][3]),
                                   pack_pair<T>(s[1][0], s[1][1]), pack_pair<T>(s[1][2], s[1][3])};
#pragma unroll
            for (int y = 0; y < VC; ++y) {
                const uint32_t *v0 = &vr[0][y].x, *v1 = &vr[1][y].x, *v2 = &vr[2][y].x, *v3 = &vr[3][y].x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mma_16x8x16<T>(o[8 * y + 2 * e], w, __byte_perm(v0[e], v1[e], 0x5410), __byte_perm(v2[e], v3[e], 0x5410));
                    mma_16x8x16<T>(o[8 * y + 2 * e + 1], w, __byte_perm(v0[e], v1[e], 0x7632), __byte_perm(v2[e], v3[e], 0x7632));
                }
            }
            load_v(n + kWarps * kKeys);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) {
                sm[warp][g + 8 * r] = top[r];
                sl[warp][g + 8 * r] = l[r];
            }
        }
        // column 2 t + j % 2 of product 8 y + e is value 8 (2 t + j % 2) + 64 y + e of the head
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) so[warp][g + 8 * (j / 2)][8 * (2 * t + j % 2) + 64 * (i / 8) + i % 8] = o[i][j];
        __syncthreads();
        for (int i = threadIdx.x; i < rows * HD; i += kWarps * 32) {
            const int r = i / HD, e = i % HD;
            float m = sm[0][r];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm[w][r]);
            float sum = 0.f, v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm[w][r] == -INFINITY ? (sl[w][r] == 0.f ? 0.f : 1.f) : exp2_fast(sm[w][r] - m);
                sum += sl[w][r] * f;
                v += so[w][r][e] * f;
            }
            if (e >= a.d) continue;
            const int h = h0 + r;
            if (p.chunks == 1) {
                row_of<T>(a.o, b, 0, h)[e] = Elem<T>::from_float(len > 0 ? v / sum : 0.f);
            } else {
                float *to = p.part + ((int64_t(b) * a.hq + h) * p.chunks + chunk) * (a.d + 2);
                to[2 + e] = v;
                if (e == 0) {
                    to[0] = sum;
                    to[1] = m;
                }
            }
        }
        __syncthreads();
    }
}

// The chunks' parts of one query head, in their order.
template <class T> __global__ void __launch_bounds__(128) decode_join_kernel(const __grid_constant__ DecodeArgs p) {
    const AttentionArgs &a = p.a;
    grid_dependency();
    const int h = int(blockIdx.x) % a.hq, b = int(blockIdx.x) / a.hq, e = threadIdx.x;
    const int len = max(0, min(a.sk, p.lengths[b]));
    const Sees see = keys_of(a, len - 1);
    const int seen = see.first_end + len - see.last, parts = (seen + p.chunk - 1) / p.chunk;
    const float *from = p.part + int64_t(blockIdx.x) * p.chunks * (a.d + 2);
    float m = -INFINITY;
    for (int i = 0; i < parts; ++i) m = fmaxf(m, from[int64_t(i) * (a.d + 2) + 1]);
    float sum = 0.f, v = 0.f;
    for (int i = 0; i < parts; ++i) {
        const float *x = from + int64_t(i) * (a.d + 2);
        const float f = x[1] == -INFINITY ? 0.f : exp2_fast(x[1] - m);
        sum += x[0] * f;
        if (e < a.d) v += x[2 + e] * f;
    }
    if (e < a.d) row_of<T>(a.o, b, 0, h)[e] = Elem<T>::from_float(len > 0 ? v / sum : 0.f);
}

// Keys of a chunk: enough CTAs to fill the GPU a few times over, since sequences differ
// in length, and 128 at least, which is two turns of a CTA's warps.
DecodeArgs plan(const AttentionArgs &a) {
    DecodeArgs p = {};
    p.a = a;
    p.row_blocks = int(ceil_div(a.group, kRows));
    const int64_t most = std::min<int64_t>(a.sk, int64_t(a.window) + a.sinks);       // keys that a token can see
    const int64_t heads = std::max<int64_t>(1, int64_t(a.batch) * a.hkv * p.row_blocks);
    const int64_t want = ceil_div(152 * 8, heads);
    int64_t chunk = ceil_div(std::max<int64_t>(1, ceil_div(most, want)), kWarps * kKeys) * kWarps * kKeys;
    chunk = std::min<int64_t>(std::max<int64_t>(chunk, 128), 512);
    p.chunk = int(chunk);
    p.chunks = int(std::max<int64_t>(1, ceil_div(most, chunk)));
    return p;
}

template <class T> basp_status go(const DecodeArgs &p, cudaStream_t stream) {
    const AttentionArgs &a = p.a;
    const dim3 grid(unsigned(p.chunks), unsigned(a.hkv * p.row_blocks), unsigned(std::min(a.batch, 65535)));
    const basp_status st = a.d <= 64 ? launch(decode_kernel<T, 64>, grid, dim3(kWarps * 32), 0, 1, stream, p)
                                     : launch(decode_kernel<T, 128>, grid, dim3(kWarps * 32), 0, 1, stream, p);
    if (st != BASP_OK || p.chunks == 1) return st;
    return launch(decode_join_kernel<T>, dim3(unsigned(a.batch * a.hq)), dim3(128), 0, 1, stream, p);
}

}  // namespace

int64_t decode_workspace(const AttentionArgs &a) {
    const DecodeArgs p = plan(a);
    return p.chunks == 1 ? 0 : int64_t(a.batch) * a.hq * p.chunks * (a.d + 2) * int64_t(sizeof(float));
}

bool decode_fits(const AttentionArgs &a) { return int64_t(a.hkv) * ceil_div(a.group, kRows) <= 65535; }

basp_status launch_attention_decode(const AttentionArgs &a, const int32_t *lengths, void *workspace, bool bf16,
                                    cudaStream_t stream) {
    DecodeArgs p = plan(a);
    p.lengths = lengths;
    p.part = static_cast<float *>(workspace);
    return bf16 ? go<__nv_bfloat16>(p, stream) : go<__half>(p, stream);
}

}  // namespace basp_fp8
