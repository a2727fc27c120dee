// attention.cuh -- the attention's kernels as attention.cu calls them.
#pragma once

#include <cuda.h>

#include "attention_common.cuh"

namespace basp_fp8 {

// Tensors as TMA sees them: boxes of 64 values x 128 rows of one head of one sequence.
// A head's or a sequence's number counts as it is (1) or not at all (0, a stride of 0).
struct HeadMaps {
    CUtensorMap q, k, v, d_o;
    int q_head, q_batch, k_head, k_batch, v_head, v_batch, do_head, do_batch;
    unsigned long long *timeouts;
};

// One token over a cache: the bytes of its workspace, and whether a grid holds its key heads.
int64_t decode_workspace(const AttentionArgs &a);
bool decode_fits(const AttentionArgs &a);
basp_status launch_attention_decode(const AttentionArgs &a, const int32_t *lengths, void *workspace, bool bf16,
                                    cudaStream_t stream);
// Key tiles whose work, for dk and dv, several CTAs share: the first `tiles`, parts first[t]
// to first[t + 1] of tile t with `chunk` pairs of tiles each.  The parts' sums pass through
// `partial`, [part][key heads of all sequences][dv, dk][128][64 or 128], and with them in `past`,
// [part][key heads of all sequences], whether something can have been past fp16's range.
constexpr int kMostSplit = 64;
struct KeySplit {
    int tiles, chunk, first[kMostSplit + 1];
    float *partial;
    uint32_t *past;
};
KeySplit key_split(const AttentionArgs &a);
int64_t key_split_parts(const AttentionArgs &a, const KeySplit &s);
int64_t key_split_bytes(const AttentionArgs &a, const KeySplit &s);
basp_status launch_attention_backward(const AttentionArgs &a, const HeadMaps &m, const KeySplit &s, bool bf16,
                                      cudaStream_t stream);
basp_status launch_attention_forward(const AttentionArgs &a, const HeadMaps &m, bool bf16, cudaStream_t stream);

}  // namespace basp_fp8
