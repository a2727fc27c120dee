// matmul.cu -- C = A B^T of two e4m3 matrices with a power-of-two scale for
// each 128 values along K (basp_matmul_fp8).
//
//     C[m][n] = sum over k of 2^(ea[m][k/128] + eb[n][k/128]) * A[m][k] * B[n][k]
//
// The tensor cores of sm_103a take such scales as they are (tcgen05.mma,
// kind::mxf8f6f4: one e8m0 byte for each row and 32 values of K, read from
// tensor memory), so a block of 128 is four instructions that name the same
// byte, and the scales cost no arithmetic.  Their 32-bit words hold four
// bytes: the scales of 512 values of K, loaded once for four blocks.
//
// Orientation.  The instruction's 128-row side is B (a weight's output
// features) and its N side, 16 to 256 wide, is A (the tokens).  The
// accumulator then has n along tensor-memory lanes and m along columns, so
// for each m a warp's 32 lanes store 32 neighbouring elements of C's row:
// coalesced whatever the row stride, the bias is one value a thread, and one
// token costs a 16-wide instruction instead of a padded 128-row one.
//
// Up to eight tokens against a B of ordinary size have a kernel of their own
// (matvec.cuh).
//
// A CTA's warps.  0 issues TMA loads (in the 128-byte swizzle; a stage is 256
// values of K, 128 in a pair).  One thread of 1 issues the products, all of its
// loop inside one election.  2 copies scales to shared memory, 3 passes them on
// to the products: a fence waits for its own warp's copies, so one warp for both
// cost 3000 cycles for each four blocks.  Four or eight more drain accumulators.
// Large products run a persistent CTA per SM, or a pair of CTAs (cta_group::2, each
// loading half of A's rows), whose accumulator is double-buffered, so a tile's
// drain overlaps the next tile's products.  With few tiles, a cluster of CTAs
// splits K; the parts meet in shared memory and are added in rank order, so
// results do not depend on timing.
//
// What bounds it.  32768 x 6144 x 2048 takes 255 to 265 us (3.1 to 3.2 PFLOP/s),
// 211 at twice the measured bf16 rate: loads from L2 (57 to 68 bytes a cycle and
// SM, each operand byte read once a tile) and, over seconds, the power limit (300
// us).  A pair reads a third less of L2 than CTAs 128 wide do, which took 298 us.
// Small products take 5 us (64 x 2048 x 2048, 0.7 of it the bytes): a launch,
// barriers, one trip to memory, a drain.
//
// Drain.  16-bit results leave tensor memory as matrix fragments, which
// stmatrix transposes into 64-byte rows of C in shared memory, and TMA stores
// them: about two instructions a value, where one store a value kept the
// products waiting (2.2 PFLOP/s at 32768 x 6144 x 2048).  TMA gets whole 16 bytes
// of a row only: a store clipped at an odd column wrote the element past it.  Up
// to seven columns at a row's end, rows of C that TMA cannot address, and
// accumulation into C take one store a value (32768 x 6143 x 2048: 291 us, 275 with
// rows at multiples of 16 bytes).  Accumulation into 16-bit C reads it value by
// value between the stores and is far from what it could be: 4.9 ms at 32768 x 6144
// x 2048, 444 us at 6144 x 2048 x 32768 (270 into 32-bit C).
//
// Long sums.  The tensor cores' 32-bit accumulator truncates: after 1024
// instructions (K = 32768) results are off by 8e-6 of themselves (in norm),
// systematically.
// For 32-bit results the accumulator therefore starts afresh every 2048
// values of K, and the drain adds the segments in registers, rounding to
// nearest (2.5e-7).  A 16-bit result's own rounding, up to 2^-11 of it in fp16, is
// sixty times larger, so there one accumulator takes all of K.
//
// Waits.  Every wait on an mbarrier has a time limit.  When one runs out the
// CTA's roles leave their loops, wait (with the limit again) for copies and
// products in flight, write NaN where results would have gone, and count it.
#include <algorithm>
#include <atomic>

#include "fp8_common.cuh"
#include "matmul_plan.h"
#include "matvec.cuh"
#include "tcgen05.cuh"

namespace basp_fp8 {
namespace {

__device__ unsigned long long g_timeouts;

constexpr uint64_t kWaitLimitNs = 2000000000ull;

constexpr int kScaleSlots = 4;           // scale words on their way, of four blocks each

// Blocks of K of a segment of a 32-bit result.
constexpr int kSegment = 16;

// Drain warps: 32-bit results keep a tile's sums in registers (128 a thread).
template <class T> __host__ __device__ constexpr int drain_warps() { return sizeof(T) == 4 ? 8 : 4; }
template <class T> __host__ __device__ constexpr int cta_threads() { return 128 + 32 * drain_warps<T>(); }
constexpr int kOutBytes = 32 * 64;       // 32 rows of 32 16-bit results
constexpr int kOutAlign = 8;             // 16-bit results of the 16 bytes that TMA stores are made of

constexpr int kSmemLimit = 227 * 1024;
constexpr int kBarrierBytes = 512;

// Sizes of a CTA whose tile is BN rows of A wide; CG = 2: of each CTA of a
// pair, which loads half of those rows.
template <int BN, int CG, class T> struct Sizes {
    static constexpr int kBlocks = stage_blocks<CG>();
    static constexpr int kRowsQ = BN / CG;
    static constexpr int kBlockP = kTileP * kBlock;            // bytes of one block of a stage
    static constexpr int kBlockQ = kRowsQ * kBlock;
    static constexpr int kStage = kBlocks * (kBlockP + kBlockQ);
    // scales of 128 rows x 4 blocks are 512 bytes; B's 128 rows, then A's BN
    static constexpr int kScale = 512 + (BN > 128 ? 1024 : 512);
    static constexpr int kScaleColumns = kScale / 128;
    // results on their way out, one or two buffers for each of four drain warps
    static constexpr int kOutBuffers = BN > 192 ? 1 : 2;   // a seventh stage is worth more
    static constexpr int kOut = sizeof(T) == 4 ? 0 : 4 * kOutBuffers * kOutBytes;
    static constexpr int kFixed = 1024 + kOut + kScaleSlots * kScale + kBarrierBytes;
    static constexpr int kStages = (kSmemLimit - kFixed) / kStage;
    static constexpr int kSmem = kFixed + kStages * kStage;
    // Tensor-memory columns: two accumulators and the scale slots.
    static constexpr int kScaleBase = 2 * BN;
    static constexpr int kNeed = kScaleBase + kScaleSlots * kScaleColumns;
    static constexpr int kColumns = kNeed <= 64 ? 64 : kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
    static constexpr int kBarriers = 2 * kStages + 3 * kScaleSlots + 5;
    static_assert(kNeed <= 512, "tensor memory");
    static_assert(8 * kBarriers + 8 <= kBarrierBytes, "barriers");
    static_assert(kBlockQ % 1024 == 0, "swizzle");
};

struct MatmulArgs {
    const uint8_t *sp, *sq;              // scales of B (P side) and A (Q side)
    int64_t sp_pitch, sq_pitch;
    int sp_shift, sq_shift;              // row -> scale row: 0 or 7
    void *c;
    const void *bias;
    int64_t c_stride;
    int M, N, nk;                        // nk: blocks of 128 along K
    int ns;                              // stages along K
    int tiles_m, tiles_n, tiles;
    int split;                           // CTAs of a cluster that share a tile
    int accumulate;
    int tma_out;                         // C's rows can be stored by TMA
};

// Tiles of one group of 16 tile rows of B run side by side over all of A, so
// what the CTAs in flight read of B stays in L2.
constexpr int kGroupN = 16;
__device__ __forceinline__ void tile_at(const MatmulArgs &a, int t, int *tm, int *tn) {
    const int per_group = kGroupN * a.tiles_m;
    const int g = t / per_group, r = t % per_group;
    const int width = min(kGroupN, a.tiles_n - g * kGroupN);
    *tn = g * kGroupN + r % width;
    *tm = r / width;
}

struct Waiter {
    volatile int *abort;                 // shared by the CTA
    template <bool CLUSTER = false>
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, bool give_up_early = true) const {
        if (mbar_try_wait<CLUSTER>(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait<CLUSTER>(bar, parity)) {
            if (give_up_early && *abort) return false;
            if (global_ns() - t0 > kWaitLimitNs) {
                if (!*abort) atomicAdd(&g_timeouts, 1ull);
                *abort = 1;
                return false;
            }
        }
        return true;
    }
    // for an arrival that may come from the other CTA's threads of a pair
    template <int CG> __device__ __forceinline__ bool pair(uint32_t bar, uint32_t parity) const {
        return operator()<CG == 2>(bar, parity);
    }
};

// A ring's place and the parity of its turn, counted instead of divided.
template <int N> struct Ring {
    uint32_t at = 0, turn = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) {
            at = 0;
            turn ^= 1;
        }
    }
};

template <class T>
__device__ __forceinline__ void put(const MatmulArgs &a, T *c, float v) {
    if (a.accumulate) v += Elem<T>::to_float(*c);
    *c = Elem<T>::from_float(v);
}

template <class T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Adds a tile's parts of all CTAs of the cluster, in rank order; each CTA
// stores a share of the columns.  `part0`: [BN][128] floats in every CTA.
template <int BN, class T>
__device__ __forceinline__ void join_parts(const MatmulArgs &a, uint32_t part0, int rank, int tm, int tn) {
    const int row = threadIdx.x % kTileP, half = threadIdx.x / kTileP, halves = blockDim.x / kTileP;
    const int64_t n = int64_t(tn) * kTileP + row, m0 = int64_t(tm) * BN;
    if (n >= a.N) return;
    const float bias = a.bias != nullptr ? Elem<T>::to_float(static_cast<const T *>(a.bias)[n]) : 0.f;
    const int j1 = min(BN * (rank + 1) / a.split, int(min(int64_t(BN), a.M - m0)));
    constexpr int U = 4;                                  // columns at once: a load takes a microsecond
    for (int j = BN * rank / a.split + half; j < j1; j += U * halves) {
        float v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) {
            if (r >= a.split) break;
            const uint32_t part = cluster_addr(part0 + uint32_t(j * kTileP + row) * 4, r);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u * halves < j1) v[u] += cluster_load(part + uint32_t(u * halves * kTileP) * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * halves < j1)
                put<T>(a, static_cast<T *>(a.c) + (m0 + j + u * halves) * a.c_stride + n, v[u] + bias);
    }
}

template <int BN, int CG, class T>
__global__ void __launch_bounds__(cta_threads<T>(), 1)
matmul_kernel(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_p,
              const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c) {
    using S = Sizes<BN, CG, T>;
    constexpr int ST = S::kStages, DW = drain_warps<T>(), SB = S::kBlocks;
    constexpr int WS = 4 / SB;                            // stages of a word of scales
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (1024 - (smem_addr(smem_raw) & 1023)) % 1024;
    uint8_t *out_smem = smem + ST * S::kStage;
    uint8_t *scale_smem = out_smem + S::kOut;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scale_smem + kScaleSlots * S::kScale);
    const uint32_t stage0 = smem_addr(smem), scale0 = smem_addr(scale_smem);
    const uint32_t full = smem_addr(bars), empty = full + 8 * ST;
    const uint32_t sfull = empty + 8 * ST, sempty = sfull + 8 * kScaleSlots;
    const uint32_t swritten = sempty + 8 * kScaleSlots;
    const uint32_t acc_full = swritten + 8 * kScaleSlots, acc_free = acc_full + 16, drained = acc_free + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::kBarriers);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // CTAs that share a tile: a pair, or the parts of a split K
    const int sharing = CG == 2 ? 2 : a.split;
    const int peer = CG == 2 ? int(blockIdx.x) % 2 : 0;    // 0 leads the pair
    const int rank = CG == 1 && a.split > 1 ? int(blockIdx.x) % a.split : 0;
    const int first = int(blockIdx.x) / sharing, step = int(gridDim.x) / sharing;
    const int s0 = int(int64_t(a.ns) * rank / a.split), s1 = int(int64_t(a.ns) * (rank + 1) / a.split);
    // one accumulator takes `segment` stages; a tile has `segments`
    const int segment = sizeof(T) == 4 ? kSegment / SB : a.ns;
    const int segments = (s1 - s0 + segment - 1) / segment;

    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&map_p);
        tma_prefetch_map(&map_q);
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < kScaleSlots; ++s) {
            mbar_init(sfull + 8 * s, CG);
            mbar_init(sempty + 8 * s, 1);
            mbar_init(swritten + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_free + 8 * s, CG * DW);
        }
        mbar_init(drained, 1);
        *abort = 0;
        fence_mbar_init();
        fence_async_shared();
    }
    if (warp == 3) tmem_alloc<CG>(smem_addr(tmem_slot), S::kColumns);
    tcgen05_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync();                          // the other CTA's barriers are there
    tcgen05_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency();
    // the leader's barriers that the other CTA's loads, scales and drains reach
    const uint32_t lead_full = CG == 2 ? cluster_addr(full, 0) : full;
    const uint32_t lead_sfull = CG == 2 ? cluster_addr(sfull, 0) : sfull;
    const uint32_t lead_acc_free = CG == 2 ? cluster_addr(acc_free, 0) : acc_free;
    auto arrive = [](uint32_t bar) {
        if constexpr (CG == 2) mbar_arrive_cluster(bar);
        else mbar_arrive(bar);
    };
    const Waiter wait{abort};

    if (warp == 0) {                                      // loads
        Ring<ST> ring;
        uint32_t issued = 0;
        bool ok = true;
        for (int t = first; t < a.tiles && ok; t += step) {
            int tm, tn;
            tile_at(a, t, &tm, &tn);
            const int p = (tn * CG + peer) * kTileP, q = tm * BN + peer * S::kRowsQ;
            for (int s = s0; s < s1; ++s, ring.next(), ++issued) {
                ok = __all_sync(0xffffffffu, wait(empty + 8 * ring.at, ring.turn ^ 1));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t to = stage0 + ring.at * S::kStage, bar = full + 8 * ring.at;
                    const int kb = s * SB, blocks = min(SB, a.nk - kb);
                    // the leader's barrier counts both CTAs' bytes
                    if (peer == 0) mbar_expect_tx(bar, CG * blocks * (S::kBlockP + S::kBlockQ));
#pragma unroll
                    for (int i = 0; i < SB; ++i) {
                        if (i >= blocks) break;
                        const uint32_t to_p = to + i * S::kBlockP;
                        const uint32_t to_q = to + SB * S::kBlockP + i * S::kBlockQ;
                        const int x = (kb + i) * kBlock;
                        if constexpr (CG == 2) {
                            tma_load_2d_pair(to_p, &map_p, x, p, lead_full + 8 * ring.at);
                            tma_load_2d_pair(to_q, &map_q, x, q, lead_full + 8 * ring.at);
                        } else {
                            tma_load_2d(to_p, &map_p, x, p, bar);
                            tma_load_2d(to_q, &map_q, x, q, bar);
                        }
                    }
                }
                __syncwarp();
            }
        }
        // A CTA ends after the last arrival at its barriers, and after its
        // copies in flight (a pair's count at the leader): also where another
        // warp gave up on them after this one had issued them all.
        const uint32_t open = issued < uint32_t(ST) ? issued : ST;
        for (uint32_t j = issued - open; j < issued; ++j) {
            if (CG == 2 && ok) wait(empty + 8 * (j % ST), (j / ST) & 1);
            if (peer == 0) wait(full + 8 * (j % ST), (j / ST) & 1, false);
        }
    } else if (warp == 1) {
        if (peer == 0 && elect_one()) {                   // products
            Ring<ST> ring;
            Ring<kScaleSlots> words;
            Ring<2> accs;
            uint32_t count = 0;
            bool ok = true, ready = false;
            for (int t = first; t < a.tiles && ok; t += step) {
                int left = 0;                             // stages left of the segment
                for (int s = s0; s < s1; ++s) {
                    const bool fresh = left == 0;
                    const bool scales = s == s0 || s % WS == 0;  // a new word: four blocks
                    if (fresh) {
                        left = segment;
                        // drained of the sum before the last
                        if (count >= 2) ok = wait.template pair<CG>(acc_free + 8 * accs.at, accs.turn ^ 1);
                    }
                    if (scales) ok = ok && wait.template pair<CG>(sfull + 8 * words.at, words.turn);
                    if (!ready) ok = ok && wait(full + 8 * ring.at, ring.turn);
                    if (!ok) break;
                    tcgen05_after_sync();
                    const uint32_t at = ring.at;
                    ring.next();
                    ready = mbar_test(full + 8 * ring.at, ring.turn);   // known by the time it is asked
                    const bool last = --left == 0 || s + 1 == s1, word_done = s + 1 == s1 || s % WS == WS - 1;
                    const uint32_t sf = tmem + S::kScaleBase + words.at * S::kScaleColumns;
                    if (scales) {
                        const uint64_t src = scale_desc(scale0 + words.at * S::kScale);
#pragma unroll
                        for (int i = 0; i < S::kScale / 512; ++i) tmem_copy_scales<CG>(sf + 4 * i, src + 32 * i);
                    }
                    const uint32_t acc = tmem + accs.at * BN;
                    const uint32_t dp = operand_desc_low(stage0) + at * (S::kStage / 16);
                    const uint32_t dq = dp + SB * S::kBlockP / 16;
                    const uint32_t idesc = mma_desc(CG * kTileP, BN) | mma_scale_ids(s % WS * SB);
#pragma unroll
                    for (int i = 0; i < SB; ++i) {
                        if (i > 0 && s * SB + i >= a.nk) break;
#pragma unroll
                        for (int k = 0; k < kBlock / 32; ++k)
                            mma_mxf8<CG>(acc, dp + i * (S::kBlockP / 16) + 2 * k, dq + i * (S::kBlockQ / 16) + 2 * k,
                                         idesc + mma_scale_ids(i), sf, sf + 4, !fresh || i > 0 || k > 0);
                    }
                    mma_commit<CG>(empty + 8 * at);
                    if (word_done) mma_commit<CG>(sempty + 8 * words.at);
                    if (last) mma_commit<CG>(acc_full + 8 * accs.at);
                    if (word_done) words.next();
                    if (last) {
                        left = 0;
                        ++count;
                        accs.next();
                    }
                }
            }
            if (!ok) {                                    // products in flight end before the CTA does
                mma_commit<CG>(drained);
                wait(drained, 0, false);
            }
        }
    } else if (warp == 2) {                               // scales
        // Each lane copies the words (four blocks' bytes) of rows lane, lane + 32,
        // ... of B's 128 and of A's to where the products' copy expects them.
        // kAhead words are on their way beside the one that is passed on: next
        // to the tiles' traffic a load takes longer than four blocks' products.
        constexpr int A = S::kScale / 512, kAhead = 1;    // A: groups of 128 rows
        static_assert(kAhead < kScaleSlots, "a slot each");
        Ring<kScaleSlots> words, passed;
        uint32_t issued = 0;
        bool ok = true;
        const int g0 = s0 / WS, g1 = (s1 + WS - 1) / WS;
        auto pass_on = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(swritten + 8 * passed.at);
            passed.next();
        };
        for (int t = first; t < a.tiles && ok; t += step) {
            int tm, tn;
            tile_at(a, t, &tm, &tn);
            const uint8_t *at[A][4];
#pragma unroll
            for (int i = 0; i < A; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int in_tile = (i > 0 ? (i - 1) * 128 : 0) + 32 * j + lane;
                    const int64_t row = i == 0 ? (int64_t(tn) * CG + peer) * kTileP + in_tile
                                               : int64_t(tm) * BN + in_tile;
                    at[i][j] = nullptr;                   // rows that do not exist: their values are 0
                    if (i == 0 && row < a.N) at[i][j] = a.sp + (row >> a.sp_shift) * a.sp_pitch;
                    if (i > 0 && in_tile < BN && row < a.M) at[i][j] = a.sq + (row >> a.sq_shift) * a.sq_pitch;
                }
            for (int g = g0; g < g1; ++g) {
                ok = __all_sync(0xffffffffu, wait(sempty + 8 * words.at, words.turn ^ 1));
                if (!ok) break;
                const uint32_t to = scale0 + words.at * S::kScale + 16 * lane;
                const int bytes = min(4, a.nk - 4 * g);   // what follows a row's last is not its
#pragma unroll
                for (int i = 0; i < A; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool have = at[i][j] != nullptr;
                        copy4_async(to + 512 * i + 4 * j, have ? at[i][j] + 4 * g : a.sp, have ? bytes : 0);
                    }
                copy_commit();
                words.next();
                if (++issued > kAhead) {
                    copy_wait<kAhead>();
                    pass_on();
                }
            }
        }
        copy_wait<0>();
        for (uint32_t j = issued < kAhead ? 0 : issued - kAhead; j < issued; ++j) pass_on();
        if (CG == 2 && ok)                                // the last arrivals, as above
            for (uint32_t j = issued < kScaleSlots ? 0 : issued - kScaleSlots; j < issued; ++j)
                wait(sempty + 8 * (j % kScaleSlots), (j / kScaleSlots) & 1);
    } else if (warp == 3) {                               // scales, on to the products
        // A warp of its own: a fence waits for the copies that its warp has in
        // flight (3000 cycles for four blocks, when one warp did both).
        Ring<kScaleSlots> words;
        bool ok = true;
        for (int t = first; t < a.tiles && ok; t += step)
            for (int g = s0 / WS; g < (s1 + WS - 1) / WS; ++g, words.next()) {
                ok = __all_sync(0xffffffffu, wait(swritten + 8 * words.at, words.turn));
                if (!ok) break;
                fence_async_shared();
                if (lane == 0) arrive(lead_sfull + 8 * words.at);
            }
    } else if (warp >= 4) {                               // drain
        const int quarter = warp % 4, row = quarter * 32 + lane;
        const uint32_t lanes = uint32_t(quarter * 32) << 16;
        float *part = reinterpret_cast<float *>(smem);     // [BN][128], split only
        Ring<2> accs;
        using Out = OutRing<S::kOutBuffers>;
        Out out;                                           // goes on from tile to tile
        bool ok = true;
        auto next_accumulator = [&]() {
            ok = __all_sync(0xffffffffu, ok && wait(acc_full + 8 * accs.at, accs.turn));
            tcgen05_after_sync();
            return tmem + lanes + accs.at * BN;
        };
        // what this warp reads of the accumulator is behind it
        auto release = [&]() {
            tcgen05_before_sync();
            __syncwarp();
            if (ok && lane == 0) arrive(lead_acc_free + 8 * accs.at);
            accs.next();
        };
        for (int t = first; t < a.tiles; t += step) {
            int tm, tn;
            tile_at(a, t, &tm, &tn);
            const int64_t n0 = (int64_t(tn) * CG + peer) * kTileP, n = n0 + row, m0 = int64_t(tm) * BN;
            const bool mine = n < a.N;
            T *c = static_cast<T *>(a.c) + m0 * a.c_stride + n;
            const float bias = mine && a.bias != nullptr && a.split == 1
                                   ? Elem<T>::to_float(static_cast<const T *>(a.bias)[n]) : 0.f;
            if constexpr (sizeof(T) == 4) {
                // Two warps a quarter, half of the columns each.
                constexpr int NC = BN < 32 ? 1 : BN / 32; // chunks of 16 columns
                const int half = (warp - 4) / 4, j0 = BN < 32 ? 0 : half * (BN / 2);
                const bool active = BN >= 32 || half == 0;
                float sum[NC][16];
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[i][j] = 0.f;
                for (int s = 0; s < segments; ++s) {
                    const uint32_t acc = next_accumulator();
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        uint32_t v[16];
                        if (ok) {
                            tmem_load16(acc + j0 + 16 * i, v);
                            tmem_load_wait();
                            tmem_loaded(v);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = 0x7fffffffu;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] += __uint_as_float(v[j]);
                    }
                    release();
                }
                if (a.split > 1) {
#pragma unroll
                    for (int i = 0; i < NC; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (ok && active) part[(j0 + 16 * i + j) * kTileP + row] = sum[i][j];
                } else if (mine && active) {
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        T *to = c + (j0 + 16 * i) * a.c_stride;
                        const int left = int(a.M - m0) - j0 - 16 * i;
                        if (a.accumulate) {
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += a.c_stride)
                                if (j < left) sum[i][j] += *to;
                            to = c + (j0 + 16 * i) * a.c_stride;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j, to += a.c_stride)
                            if (j < left) *to = sum[i][j] + bias;
                    }
                }
            } else if (a.tma_out) {
                // Fragments hold lanes t / 4 and t / 4 + 8 of each 16.
                float fb[2][2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int64_t k = n0 + quarter * 32 + 16 * h + 8 * q + lane / 4;
                        fb[h][q] = k < a.N && a.bias != nullptr ? Elem<T>::to_float(static_cast<const T *>(a.bias)[k])
                                                                : 0.f;
                    }
                const uint32_t acc = next_accumulator();
                constexpr int CH = BN < 32 ? 1 : BN / 32;  // chunks of 32 columns (a narrow tile: 16 used)
                const uint32_t out0 = smem_addr(out_smem) + quarter * S::kOutBuffers * kOutBytes;
                // TMA takes the warp's columns up to tma_end; up to seven more follow
                const int64_t w0 = n0 + quarter * 32, tma_end = a.N / kOutAlign * kOutAlign;
                const int tail_end = int(min(int64_t(32), a.N - w0));
                const int tail0 = int(max(int64_t(0), min(int64_t(32), tma_end - w0)));
                // row lane % 8 of matrix lane / 8: 16 bytes in the 64-byte swizzle
                const int r8 = lane % 8, piece = lane / 8;
                for (int ch = 0; ch < CH; ++ch) {
                    uint32_t v[2][16];
                    if (ok) {
                        tmem_load_fragments(acc + 32 * ch, v[0]);
                        tmem_load_fragments(acc + 32 * ch + (16u << 16), v[1]);
                        tmem_load_wait();
                        tmem_loaded(v[0]);
                        tmem_loaded(v[1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[0][j] = v[1][j] = 0x7fffffffu;
                    }
                    if (ch + 1 == CH) release();
                    const uint32_t buf = out0 + out.next() * kOutBytes;
                    if (lane == 0) tma_store_wait_read<Out::kUnread>();
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t p[2][2];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                p[h][q] = pack2<T>(__uint_as_float(v[h][4 * g + 2 * q]) + fb[h][q],
                                                   __uint_as_float(v[h][4 * g + 2 * q + 1]) + fb[h][q]);
                        const int r = 8 * g + r8;
                        store_matrix_transposed(buf + r * 64 + 16 * (piece ^ ((r >> 1) & 3)), p[0][0], p[0][1],
                                                p[1][0], p[1][1]);
                    }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (w0 < tma_end && m0 + 32 * ch < a.M)
                            tma_store_2d(&map_c, buf, int(w0), int(m0) + 32 * ch);
                        tma_store_commit();               // also of nothing: buffers are counted in groups
                    }
                    // a lane has a row of C; the buffer is written again after the next __syncwarp
                    if (tail0 < tail_end && lane < BN && m0 + 32 * ch + lane < a.M) {
                        T *to = static_cast<T *>(a.c) + (m0 + 32 * ch + lane) * a.c_stride + w0;
#pragma unroll 1
                        for (int k = tail0; k < tail_end; ++k)
                            to[k] = *reinterpret_cast<const T *>(
                                smem + (buf - stage0) + lane * 64 + 16 * (k / 8 ^ ((lane >> 1) & 3)) + k % 8 * 2);
                    }
                }
            } else {
                const uint32_t acc = next_accumulator();
                for (int j0 = 0; j0 < BN; j0 += 16) {
                    uint32_t v[16];
                    if (ok) {
                        tmem_load16(acc + j0, v);
                        tmem_load_wait();
                        tmem_loaded(v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = 0x7fffffffu;
                    }
                    if (j0 + 16 == BN) release();
                    if (a.split > 1) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (ok) part[(j0 + j) * kTileP + row] = __uint_as_float(v[j]);
                    } else if (mine) {
                        T *to = c + j0 * a.c_stride;
                        if (!a.accumulate && m0 + j0 + 16 <= a.M) {
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += a.c_stride)
                                *to = Elem<T>::from_float(__uint_as_float(v[j]) + bias);
                        } else {
#pragma unroll
                            for (int j = 0; j < 16; ++j, to += a.c_stride)
                                if (m0 + j0 + j < a.M) put<T>(a, to, __uint_as_float(v[j]) + bias);
                        }
                    }
                }
            }
        }
        if (a.tma_out && lane == 0) tma_store_wait_read<0>();   // shared memory stays until it is read
    }

    if (CG == 1 && a.split > 1) {                         // one tile: join the cluster's parts
        __syncthreads();
        if (*abort)                                       // nothing is in flight any more
            for (int i = threadIdx.x; i < BN * kTileP; i += blockDim.x)
                reinterpret_cast<uint32_t *>(smem)[i] = 0x7fffffffu;
        __syncwarp();
        cluster_sync();
        int tm, tn;
        tile_at(a, first, &tm, &tn);
        join_parts<BN, T>(a, stage0, rank, tm, tn);
        __syncwarp();
        cluster_sync();                                   // the others may still read this CTA's part
    }
    tcgen05_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync();                          // nothing of the pair's reaches the other any more
    tcgen05_after_sync();
    if (warp == 3) tmem_free<CG>(tmem, S::kColumns);
}

// C = bias, zero, or itself where there is nothing to sum over.
template <class T>
__global__ void bias_kernel(const __grid_constant__ MatmulArgs a) {
    grid_dependency();
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= int64_t(a.M) * a.N) return;
    const int64_t m = i / a.N, n = i % a.N;
    put<T>(a, static_cast<T *>(a.c) + m * a.c_stride + n,
           a.bias != nullptr ? Elem<T>::to_float(static_cast<const T *>(a.bias)[n]) : 0.f);
}

// ---- host ---------------------------------------------------------------------

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

// Boxes of 128 bytes of K x `box_rows`; past the matrix' end they read zero.
bool encode(const basp_fp8_matrix *m, int box_rows, CUtensorMap *out) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {cuuint64_t(m->cols), cuuint64_t(m->rows)};
    const cuuint64_t strides[1] = {cuuint64_t(m->pitch)};
    const cuuint32_t box[2] = {kBlock, cuuint32_t(box_rows)};
    const cuuint32_t elem[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m->data, dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Boxes of 32 x 32 16-bit results of C (16 rows where tiles are that narrow), up
// to the last whole 16 bytes of its rows.
bool encode_out(const MatmulArgs &a, int box_rows, CUtensorMap *out) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {cuuint64_t(a.N / kOutAlign * kOutAlign), cuuint64_t(a.M)};
    const cuuint64_t strides[1] = {cuuint64_t(a.c_stride) * 2};
    const cuuint32_t box[2] = {32, cuuint32_t(box_rows)};
    const cuuint32_t elem[2] = {1, 1};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.c, dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int CG, class T>
basp_status launch_matmul(MatmulArgs a, const basp_fp8_matrix *p, const basp_fp8_matrix *q, int sms,
                          cudaStream_t stream) {
    CUtensorMap map_p, map_q, map_c = {};
    // one row of C: its stride is free
    if (a.M == 1) a.c_stride = ceil_div(a.N, kOutAlign) * kOutAlign;
    a.tma_out = sizeof(T) == 2 && a.split == 1 && !a.accumulate && a.N >= kOutAlign &&
                uintptr_t(a.c) % 16 == 0 && a.c_stride % kOutAlign == 0;
    if (!encode(p, kTileP, &map_p) || !encode(q, BN / CG, &map_q) ||
        (a.tma_out && !encode_out(a, BN < 32 ? BN : 32, &map_c)))
        return BASP_ERR_CUDA;
    static std::atomic<bool> ready[64];   // per device; a benign race
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BASP_ERR_CUDA;
    if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(matmul_kernel<BN, CG, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Sizes<BN, CG, T>::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return BASP_ERR_CUDA;
        }
        if (dev < 64) ready[dev].store(true, std::memory_order_release);
    }
    const int ctas = a.split > 1 ? a.tiles * a.split : std::min(a.tiles * CG, sms / CG * CG);
    return launch(matmul_kernel<BN, CG, T>, dim3(unsigned(ctas)), dim3(cta_threads<T>()), Sizes<BN, CG, T>::kSmem,
                  a.split * CG, stream, a, map_p, map_q, map_c);
}

template <class T>
basp_status run(MatmulArgs a, const basp_fp8_matrix *p, const basp_fp8_matrix *q, cudaStream_t stream) {
    if (a.nk == 0) {
        if (a.accumulate && a.bias == nullptr) return BASP_OK;
        const int64_t ctas = ceil_div(int64_t(a.M) * a.N, 256);
        if (ctas > kMaxSide) return BASP_ERR_TOO_LARGE;
        return launch(bias_kernel<T>, dim3(unsigned(ctas)), dim3(256), 0, 1, stream, a);
    }
    const int sms = sm_count();
    const Shape s = pick_shape(a.M, a.N, a.nk, sms);
    a.tiles_m = int(ceil_div(a.M, s.bn));
    a.tiles_n = int(ceil_div(a.N, kTileP * (1 + s.pair)));
    const int64_t tiles = int64_t(a.tiles_m) * a.tiles_n;
    if (tiles > (int64_t(1) << 30)) return BASP_ERR_TOO_LARGE;
    a.tiles = int(tiles);
    a.split = s.split;
    a.ns = int(ceil_div(a.nk, s.pair ? stage_blocks<2>() : stage_blocks<1>()));
    switch (s.bn) {
        case 16: return launch_matmul<16, 1, T>(a, p, q, sms, stream);
        case 32: return launch_matmul<32, 1, T>(a, p, q, sms, stream);
        case 64: return launch_matmul<64, 1, T>(a, p, q, sms, stream);
        case 128: return launch_matmul<128, 1, T>(a, p, q, sms, stream);
        case 192: return launch_matmul<192, 2, T>(a, p, q, sms, stream);
        default: return launch_matmul<224, 2, T>(a, p, q, sms, stream);
    }
}

}  // namespace
}  // namespace basp_fp8

using namespace basp_fp8;

extern "C" basp_status basp_matmul_fp8(const basp_fp8_matrix *a, const basp_fp8_matrix *b, const void *bias,
                                       int accumulate, basp_dtype dtype, void *c, int64_t c_stride,
                                       cudaStream_t stream) {
    NvtxRange range("basp_matmul_fp8");
    const int64_t esz = elem_size(dtype);
    if (esz == 0 || a == nullptr || b == nullptr || a->cols != b->cols) return BASP_ERR_INVALID_ARG;
    basp_status st = BASP_OK;
    if (!sides_ok(a->rows, a->cols, &st) || !sides_ok(b->rows, b->cols, &st)) return st;
    Args args;
    args.fp8(a, a->rows, a->cols, false);
    args.fp8(b, b->rows, b->cols, false);
    args.matrix(bias, 1, b->rows, b->rows, esz, false, false);
    args.matrix(c, a->rows, b->rows, c_stride, esz, true);
    st = args.status();
    if (st != BASP_OK || a->rows == 0 || b->rows == 0) return st;

    if (takes_matvec(a->rows, b->rows, a->cols)) {
        MatvecArgs v = {};
        v.x = static_cast<const uint8_t *>(a->data);
        v.w = static_cast<const uint8_t *>(b->data);
        v.sx = static_cast<const uint8_t *>(a->scales);
        v.sw = static_cast<const uint8_t *>(b->scales);
        v.x_pitch = a->pitch;
        v.w_pitch = b->pitch;
        v.sx_pitch = a->scale_pitch;
        v.sw_pitch = b->scale_pitch;
        v.sx_shift = a->block_rows == 1 ? 0 : 7;
        v.sw_shift = b->block_rows == 1 ? 0 : 7;
        v.c = c;
        v.bias = bias;
        v.c_stride = c_stride;
        v.M = int(a->rows);
        v.N = int(b->rows);
        v.K = int(a->cols);
        v.accumulate = accumulate != 0;
        switch (dtype) {
            case BASP_DTYPE_BF16: return launch_matvec<__nv_bfloat16>(v, stream);
            case BASP_DTYPE_FP16: return launch_matvec<__half>(v, stream);
            default: return launch_matvec<float>(v, stream);
        }
    }

    MatmulArgs m = {};
    m.sp = static_cast<const uint8_t *>(b->scales);
    m.sq = static_cast<const uint8_t *>(a->scales);
    m.sp_pitch = b->scale_pitch;
    m.sq_pitch = a->scale_pitch;
    m.sp_shift = b->block_rows == 1 ? 0 : 7;
    m.sq_shift = a->block_rows == 1 ? 0 : 7;
    m.c = c;
    m.bias = bias;
    m.c_stride = c_stride;
    m.M = int(a->rows);
    m.N = int(b->rows);
    m.nk = int(ceil_div(a->cols, kBlock));
    m.accumulate = accumulate != 0;
    switch (dtype) {
        case BASP_DTYPE_BF16: return run<__nv_bfloat16>(m, b, a, stream);
        case BASP_DTYPE_FP16: return run<__half>(m, b, a, stream);
        default: return run<float>(m, b, a, stream);
    }
}

extern "C" basp_status basp_matmul_fp8_timeouts(unsigned long long *count) {
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
