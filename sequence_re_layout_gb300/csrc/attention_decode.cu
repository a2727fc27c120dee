// attention_decode.cu -- one new token of each sequence over a cache.
//
// Memory is the bound: the visible keys and values are read once, 4 d flops for each
// 4 d bytes and query head.  A CTA has one key head of one sequence, the (up to 16) query
// heads that share it, and a chunk of the visible keys; four warps take 16 keys at a time
// in turn, each with its own running maximum and sum, and meet in shared memory at the
// end.  Where there is more than one chunk, a second kernel joins the chunks' parts in
// their order.
//
// Keys and values go through mma.sync (16 query rows x 8 keys or columns x 16): a
// tcgen05 product would want 128 rows.  Each lane copies the 16-byte pieces that it will
// read itself to shared memory, some turns ahead, so that no register holds what is on its
// way and no barrier is needed: what bounds such a kernel is the number of bytes in flight.
// One sequence of 16001 keys, 8 key heads of 64: 11.2 us (38 with the loads in registers); 32
// of up to 16384, 16 of 128, window 4096: 63.6 us, 0.66 of a copy's rate (84).
//
// The sum over a head's values may be taken in any order, so lane t of four takes the values
// 8 t + 32 c .. + 7 of a key for both operands, as they lie; for the product with V, lane g
// of eight takes the columns 8 g + 64 c .. + 7 of its four keys, and pairs of keys are put
// together by byte permutations.
#include <algorithm>

#include "attention.cuh"

namespace basp_fp8 {
namespace {

constexpr int kWarps = 4, kKeys = 16, kRows = 16;

struct DecodeArgs {
    AttentionArgs a;
    const int32_t *lengths;
    float *part;                         // [batch][Hq][chunks][d]: O
    float2 *part_stats;                  // [batch][Hq][chunks]: maximum, sum
    int chunk, chunks, row_blocks;
};

// Turns on their way, and shared memory: 128 KB or more are in flight on an SM, with two
// CTAs of heads of 128, or three of 64.
template <int HD> struct DecodeSizes {
    static constexpr int kStages = HD == 128 ? 3 : 4;
    static constexpr int kPieces = 2 * (HD / 32) + 4 * (HD / 64);      // of K and of V, a lane and turn
    static constexpr int kRing = kStages * kPieces * 32 * 16;          // bytes of a warp
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kSmem >= kWarps * kRows * (HD + 4) * 4, "the parts of the warps");
    static constexpr int kCtas = HD == 128 ? 2 : 3;
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

template <class T, int HD>
__global__ void __launch_bounds__(kWarps * 32, DecodeSizes<HD>::kCtas) decode_kernel(const __grid_constant__ DecodeArgs p) {
    constexpr int KC = HD / 32, VC = HD / 64;                 // 16-byte pieces of a key, of a value row, a lane
    constexpr int ST = DecodeSizes<HD>::kStages, PIECES = DecodeSizes<HD>::kPieces;
    extern __shared__ __align__(16) uint8_t smem[];
    float(*so)[kRows][HD + 4] = reinterpret_cast<float(*)[kRows][HD + 4]>(smem);        // at the end
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
        uint4 *mine = reinterpret_cast<uint4 *>(smem + warp * DecodeSizes<HD>::kRing) + lane;
        auto fetch = [&](int n, int stage) {
            uint4 *to = mine + stage * PIECES * 32;
            if (n < n1) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {                 // key g of each eight
                    const int i = n + 8 * x + g;
                    const T *r = kp + int64_t(i < see.first_end ? i : i + skip) * a.k.ss + 8 * t;
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const bool in = i < n1 && 8 * t + 32 * c < a.d;
                        copy16_async(to + (x * KC + c) * 32, in ? r + 32 * c : kp, in);
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {                 // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
                    const int i = n + 8 * (x / 2) + 2 * t + x % 2;
                    const T *r = vp + int64_t(i < see.first_end ? i : i + skip) * a.v.ss + 8 * g;
#pragma unroll
                    for (int c = 0; c < VC; ++c) {
                        const bool in = i < n1 && 8 * g + 64 * c < a.d;
                        copy16_async(to + (2 * KC + x * VC + c) * 32, in ? r + 64 * c : vp, in);
                    }
                }
            }
            copy_commit();                                    // an empty group past the end keeps the count
        };
        float o[HD / 8][4], top[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        const float c = a.scale * kLog2e;
        int n = n0 + warp * kKeys, stage = 0;
#pragma unroll
        for (int x = 0; x < ST - 1; ++x) fetch(n + x * kWarps * kKeys, x);
        for (; n < n1; n += kWarps * kKeys) {
            fetch(n + (ST - 1) * kWarps * kKeys, stage == 0 ? ST - 1 : stage - 1);
            copy_wait<ST - 1>();
            const uint4 *from = mine + stage * PIECES * 32;
            stage = stage + 1 < ST ? stage + 1 : 0;
            float s[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[x][j] = 0.f;
#pragma unroll
                for (int y = 0; y < KC; ++y) {
                    const uint4 k = from[(x * KC + y) * 32];
                    mma_16x8x16<T>(s[x], q[2 * y], k.x, k.y);
                    mma_16x8x16<T>(s[x], q[2 * y + 1], k.z, k.w);
                }
            }
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
                uint32_t v[4][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 u = from[(2 * KC + x * VC + y) * 32];
                    v[x][0] = u.x; v[x][1] = u.y; v[x][2] = u.z; v[x][3] = u.w;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mma_16x8x16<T>(o[8 * y + 2 * e], w, __byte_perm(v[0][e], v[1][e], 0x5410), __byte_perm(v[2][e], v[3][e], 0x5410));
                    mma_16x8x16<T>(o[8 * y + 2 * e + 1], w, __byte_perm(v[0][e], v[1][e], 0x7632), __byte_perm(v[2][e], v[3][e], 0x7632));
                }
            }
        }
        copy_wait<0>();
        __syncthreads();                                      // the rings are free
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
            for (int j = 0; j < 4; ++j)
                if (g + 8 * (j / 2) < rows) so[warp][g + 8 * (j / 2)][8 * (2 * t + j % 2) + 64 * (i / 8) + i % 8] = o[i][j];
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
                const int64_t at = (int64_t(b) * a.hq + h) * p.chunks + chunk;
                p.part[at * a.d + e] = v;
                if (e == 0) p.part_stats[at] = make_float2(m, sum);
            }
        }
        __syncthreads();
    }
}

// The chunks' parts of one query head: lanes of 16 bytes of O, several parts at a time,
// each lane's in their order and then the lanes' in theirs.
constexpr int kJoinThreads = 128;
template <class T> __global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeArgs p) {
    __shared__ float4 so[kJoinThreads];
    __shared__ float ssum[kJoinThreads / 32], smax[kJoinThreads / 32];
    const AttentionArgs &a = p.a;
    grid_dependency();
    const int h = int(blockIdx.x) % a.hq, b = int(blockIdx.x) / a.hq, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int len = max(0, min(a.sk, p.lengths[b]));
    const Sees see = keys_of(a, len - 1);
    const int seen = see.first_end + len - see.last, parts = (seen + p.chunk - 1) / p.chunk;
    const float2 *stats = p.part_stats + int64_t(blockIdx.x) * p.chunks;
    const float4 *part = reinterpret_cast<const float4 *>(p.part + int64_t(blockIdx.x) * p.chunks * a.d);
    // what a lane needs first, all on its way before anything is waited for
    constexpr int kFirst = 8;
    const int quads = a.d / 4, slices = kJoinThreads / quads, slice = tid / quads, e = tid % quads;
    float2 ahead_stats[kFirst];
    float4 ahead[kFirst];
#pragma unroll
    for (int x = 0; x < kFirst; ++x) {
        const int i = slice + x * slices;
        const bool in = slice < slices && i < parts;
        ahead_stats[x] = in ? stats[i] : make_float2(-INFINITY, 0.f);
        ahead[x] = in ? part[int64_t(i) * quads + e] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = -INFINITY, sum = 0.f;
    for (int i = tid; i < parts; i += kJoinThreads) {
        const float2 x = stats[i];
        const float top = fmaxf(m, x.x);
        // a part of nothing but minus infinities has a sum of 0, or of NaN
        sum = sum * (m == -INFINITY ? 1.f : exp2_fast(m - top)) + x.y * (x.x == -INFINITY ? 1.f : exp2_fast(x.x - top));
        m = top;
    }
    float top = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    sum = warp_add(sum * (m == -INFINITY ? 1.f : exp2_fast(m - top)));
    if (lane == 0) {
        smax[warp] = top;
        ssum[warp] = sum;
    }
    __syncthreads();
    m = fmaxf(fmaxf(smax[0], smax[1]), fmaxf(smax[2], smax[3]));
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) sum += ssum[w] * (smax[w] == -INFINITY ? 1.f : exp2_fast(smax[w] - m));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float2 s, float4 x) {
        const float f = s.x == -INFINITY ? 1.f : exp2_fast(s.x - m);
        v.x = fmaf(x.x, f, v.x);
        v.y = fmaf(x.y, f, v.y);
        v.z = fmaf(x.z, f, v.z);
        v.w = fmaf(x.w, f, v.w);
    };
#pragma unroll
    for (int x = 0; x < kFirst; ++x) add(ahead_stats[x], ahead[x]);
    if (slice < slices)
        for (int i = slice + kFirst * slices; i < parts; i += slices) add(stats[i], part[int64_t(i) * quads + e]);
    so[tid] = v;
    __syncthreads();
    if (tid >= quads) return;
    for (int i = 1; i < slices; ++i) {
        const float4 x = so[i * quads + tid];
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
    }
    const float inv = 1.f / sum;
    const bool any = len > 0;
    *reinterpret_cast<uint2 *>(row_of<T>(a.o, b, 0, h) + 4 * tid) =
        make_uint2(pack_pair<T>(any ? v.x * inv : 0.f, any ? v.y * inv : 0.f),
                   pack_pair<T>(any ? v.z * inv : 0.f, any ? v.w * inv : 0.f));
}

// Keys of a chunk: as many CTAs as fit at once for one sequence, four times that for
// several, which differ in length; 128 at least (two turns of a CTA's warps), 1024 at most.
DecodeArgs plan(const AttentionArgs &a) {
    DecodeArgs p = {};
    p.a = a;
    p.row_blocks = int(ceil_div(a.group, kRows));
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(a.sk, int64_t(a.window) + a.sinks));   // that a token can see
    const int64_t heads = std::max<int64_t>(1, int64_t(a.batch) * a.hkv * p.row_blocks);
    const int64_t ctas = int64_t(kSms) * (a.d <= 64 ? DecodeSizes<64>::kCtas : DecodeSizes<128>::kCtas) * (a.batch == 1 ? 1 : 4);
    const int64_t turn = kWarps * kKeys;
    int64_t chunk = ceil_div(ceil_div(most, std::max<int64_t>(1, ctas / heads)), turn) * turn;
    chunk = std::min<int64_t>(std::max<int64_t>(chunk, 128), 1024);
    p.chunk = int(chunk);
    p.chunks = int(ceil_div(most, chunk));
    return p;
}

template <class T, int HD> basp_status go(const DecodeArgs &p, cudaStream_t stream) {
    constexpr auto kernel = decode_kernel<T, HD>;
    constexpr size_t smem = DecodeSizes<HD>::kSmem;
    if (!allow_shared_memory<kernel, smem>()) return BASP_ERR_CUDA;
    const AttentionArgs &a = p.a;
    const dim3 grid(unsigned(p.chunks), unsigned(a.hkv * p.row_blocks), unsigned(std::min(a.batch, 65535)));
    const basp_status st = launch(kernel, grid, dim3(kWarps * 32), smem, 1, stream, p);
    if (st != BASP_OK || p.chunks == 1) return st;
    return launch(decode_join_kernel<T>, dim3(unsigned(a.batch * a.hq)), dim3(kJoinThreads), 0, 1, stream, p);
}

// The parts' statistics, then O, which begins at a multiple of 16 bytes.
int64_t stats_bytes(const DecodeArgs &p) {
    return ceil_div(int64_t(p.a.batch) * p.a.hq * p.chunks * int64_t(sizeof(float2)), 16) * 16;
}

}  // namespace

int64_t decode_workspace(const AttentionArgs &a) {
    const DecodeArgs p = plan(a);
    return p.chunks == 1 ? 0 : stats_bytes(p) + int64_t(a.batch) * a.hq * p.chunks * a.d * int64_t(sizeof(float));
}

bool decode_fits(const AttentionArgs &a) { return int64_t(a.hkv) * ceil_div(a.group, kRows) <= 65535; }

basp_status launch_attention_decode(const AttentionArgs &a, const int32_t *lengths, void *workspace, bool bf16,
                                    cudaStream_t stream) {
    DecodeArgs p = plan(a);
    p.lengths = lengths;
    p.part_stats = static_cast<float2 *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + stats_bytes(p));
    if (bf16) return a.d <= 64 ? go<__nv_bfloat16, 64>(p, stream) : go<__nv_bfloat16, 128>(p, stream);
    return a.d <= 64 ? go<__half, 64>(p, stream) : go<__half, 128>(p, stream);
}

}  // namespace basp_fp8
