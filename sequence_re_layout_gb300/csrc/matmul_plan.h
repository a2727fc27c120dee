// matmul_plan.h -- the parts of matmul.cu that a host program can check
// (tests/c/matmul_plan_test.cpp).
#pragma once

#ifdef __CUDACC__
#define BASP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BASP_HOST_DEVICE inline
#endif

namespace basp_fp8 {

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
