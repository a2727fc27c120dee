// matmul_plan_test.cpp -- host test of sequence_re_layout_gb300/csrc/
// matmul_plan.h.  Test program.
//   matmul_plan_test         checks; exit status 0 and "matmul_plan ok" on success
//   matmul_plan_test SMS M N K [M N K ...]
//                            for each product: the tile's width (0: matvec.cuh),
//                            whether by pairs, the CTAs that share K, the most
//                            tiles of a CTA, and the blocks of K of one CTA
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "matmul_plan.h"

// A drain warp's TMA stores, at their slowest: a group is read out of its
// buffer only when a wait demands it.
struct Stores {
    std::vector<int> unread;                  // buffers of the groups not read yet, oldest first
    void wait_all_but(int newest) {
        while (int(unread.size()) > newest) unread.erase(unread.begin());
    }
    bool reading(int buffer) const {
        for (int b : unread)
            if (b == buffer) return true;
        return false;
    }
};

// Whether no buffer is ever written while a store may still read it, over
// `tiles` tiles of `chunks` chunks each; `pick` chooses a chunk's buffer.
template <class F> static bool safe(int tiles, int chunks, int unread, F pick) {
    Stores stores;
    for (int t = 0; t < tiles; ++t)
        for (int ch = 0; ch < chunks; ++ch) {
            const int buffer = pick(ch);
            stores.wait_all_but(unread);
            if (stores.reading(buffer)) return false;
            stores.unread.push_back(buffer);
        }
    return true;
}

template <int BUFFERS> static void check_ring() {
    for (int chunks = 1; chunks <= 9; ++chunks) {
        basp_fp8::OutRing<BUFFERS> ring;
        if (!safe(12, chunks, ring.kUnread, [&](int) { return ring.next(); })) {
            std::fprintf(stderr, "matmul_plan: %d buffers, %d chunks a tile: overwritten\n", BUFFERS, chunks);
            std::exit(1);
        }
        // counted anew for each tile, a tile of an odd number of chunks
        // starts with the buffer that the one before ended with
        const bool anew = safe(12, chunks, ring.kUnread, [&](int ch) { return ch % BUFFERS; });
        if (anew != (chunks % BUFFERS == 0)) {
            std::fprintf(stderr, "matmul_plan: the model of stores misses an overwritten buffer\n");
            std::exit(1);
        }
    }
}

static void print_plan(int sms, int64_t M, int64_t N, int64_t K) {
    using namespace basp_fp8;
    if (takes_matvec(M, N, K)) {
        std::printf("0 0 0 0 0\n");
        return;
    }
    const int64_t nk = parts_of(K, BASP_FP8_BLOCK);
    const Shape s = pick_shape(M, N, nk, sms);
    const int64_t tiles = parts_of(M, s.bn) * parts_of(N, kTileP * (1 + s.pair)), places = sms / (1 + s.pair) / s.split;
    std::printf("%d %d %d %d %d\n", s.bn, s.pair, s.split, int(parts_of(tiles, places)), int(nk / s.split));
}

int main(int argc, char **argv) {
    for (int i = 2; i + 2 < argc; i += 3)
        print_plan(std::atoi(argv[1]), std::atoll(argv[i]), std::atoll(argv[i + 1]), std::atoll(argv[i + 2]));
    if (argc > 1) return 0;
    check_ring<1>();
    check_ring<2>();
    check_ring<3>();
    std::printf("matmul_plan ok\n");
    return 0;
}
