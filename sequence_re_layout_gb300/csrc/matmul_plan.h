// matmul_plan.h -- the parts of matmul.cu that a host program can check
// (tests/c/matmul_plan_test.cpp): which kernel and tile a product gets, and in
// what order results use shared memory.
#pragma once

#include <algorithm>
#include <cstdint>

#include "basp_fp8.h"

#ifdef __CUDACC__
#define BASP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BASP_HOST_DEVICE inline
#endif

namespace basp_fp8 {

// ---- which kernel and tile ------------------------------------------------------

constexpr int kVecTokens = 8;

// Whether matvec.cuh's kernel takes the product.  GPU times in us of one and of
// eight tokens there, and of either on matmul.cu's tiles: 128 x 128 1.4, 1.4, 2.7;
// 2048 x 2048 2.5, 2.6, 5.0; 6144 x 2048 3.4, 3.6, 5.0; 8192 x 1024 3.4, 3.7, 3.9;
// 16384 x 512 3.4, 3.5, 3.5; 4096 x 4096 5.0, 5.4, 6.1; 512 x 16384 6.2, 6.5, 8.8; at
// the bounds 8191 x 2048 5.1, 5.4, 5.0 to 5.3; but past them, one token: 16384 x 1024
// 5.4, tiles 4.2; 8192 x 2048 5.3, 5.1; 16384 x 2048 10.6, 7.9.
inline bool takes_matvec(int64_t M, int64_t N, int64_t K) {
    return M <= kVecTokens && K > 0 && N * K <= (N < 8192 ? int64_t(1) << 24 : int64_t(1) << 23);
}

constexpr int kTileP = 128;              // rows of B a tile: the instruction's M
// Blocks of 128 along K of a stage.  A pair, which waits for loads more than
// for anything else, has as many stages on their way as fit; a CTA alone
// spends more on a stage's bookkeeping.
template <int CG> BASP_HOST_DEVICE constexpr int stage_blocks() { return CG == 2 ? 1 : 2; }
constexpr int kMaxSplit = 4;             // CTAs that share K: eight rarely fit a GPC at once

inline int64_t parts_of(int64_t a, int64_t part) { return (a + part - 1) / part; }

struct Shape {
    int bn, pair, split;
};

// The tile (its width along A's rows, one CTA or a pair) and the number of
// CTAs that split K with the least estimated time, in SM cycles: rounds of
// tiles over the SMs, each paying for its blocks of K, and what no round
// hides.  The figures are fits to GPU times on 152 SMs: one tile of K = 2048
// takes 5.0 us at 16 wide, 6.8 at 128, 8.7 in a pair 192 wide, and 0.15, 0.19
// and 0.20 us for each further block; beside other CTAs an SM gets 57 to 68
// bytes a cycle from L2; a split into 4 takes 6.9 us instead of 11.9 at 16 x
// 1024 x 8192, and 5.2 instead of 5.0 at 16 x 2048 x 2048.
inline Shape pick_shape(int64_t M, int64_t N, int64_t nk, int sms) {
    Shape best = {128, 0, 1};
    double best_cost = 1e300;
    auto consider = [&](int bn, int pair, int split) {
        const int cg = 1 + pair;
        const int64_t tiles = parts_of(M, bn) * parts_of(N, kTileP * cg);
        if (split > 1 && (split > parts_of(nk, stage_blocks<1>()) || tiles * split > sms)) return;
        // a block's products, its loads, or what issuing them takes
        const double block = std::max({2.0 * bn, (kTileP + bn / cg) * BASP_FP8_BLOCK / (pair ? 57.0 : 68.0), 280.0});
        const double rounds = double(parts_of(tiles * split * cg, sms));
        const double start = pair ? 9000 + 8.0 * bn : 5000 + 15.0 * bn;
        const double cost = start + rounds * double(parts_of(nk, split)) * block +
                            (split > 1 ? 3000 + 70.0 * bn : 0);
        if (cost < best_cost) {
            best_cost = cost;
            best = {bn, pair, split};
        }
    };
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (bn > 16 && bn / 2 >= M) break;
        for (int split = 1; split <= kMaxSplit; split *= 2) consider(bn, 0, split);
    }
    if (M > 128)
        for (int bn : {224, 192}) consider(bn, 1, 1);
    return best;
}

// ---- results on their way out ---------------------------------------------------

// The buffers from which a drain warp stores its results (TMA stores), taken in
// turn over all chunks of all tiles of its CTA.  One group of stores is
// committed for each buffer taken.  Before a buffer is written, all but the
// newest kUnread groups have been read out of shared memory; the group that
// last used this buffer is the next older one, whatever a tile's number of chunks.
template <int BUFFERS> struct OutRing {
    static constexpr int kUnread = BUFFERS - 1;
    int at = 0;
    BASP_HOST_DEVICE int next() {
        const int now = at;
        at = at + 1 < BUFFERS ? at + 1 : 0;
        return now;
    }
};

}  // namespace basp_fp8
