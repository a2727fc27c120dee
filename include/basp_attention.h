/*
 * basp_attention.h -- C ABI of the attention between the two re-layouts (same
 * library, libbasp.so, and same conventions as basp.h and basp_fp8.h).
 *
 * Causal attention with a sliding window and a few first tokens that stay visible
 * (sinks).  Query i of Sq stands at position p = i + Sk - Sq among the Sk keys, so
 * Sq = Sk is a whole sequence and Sq < Sk a piece of one behind a cache.  It sees
 * key j if
 *     j <= p  and  (j > p - window  or  j < sinks).
 * With s_ij = scale * q_i . k_j over the keys that i sees,
 *     lse_i = log sum_j exp(s_ij),  P_ij = exp(s_ij - lse_i),  o_i = sum_j P_ij v_j.
 * A query that sees nothing (Sq > Sk) has o = 0 and lse = minus infinity.  What a
 * query does not see has no part in its results, also where it is infinite or NaN.
 *
 * Gradients, with dP_ij = do_i . v_j and D_i = do_i . o_i:
 *     dS_ij = P_ij (dP_ij - D_i),   dq_i = scale * sum_j dS_ij k_j,
 *     dk_j = scale * sum_i dS_ij q_i,   dv_j = sum_i P_ij do_i,
 * dk and dv summed over the Hq / Hkv query heads that share a key head.
 *
 * Products are of 16-bit values, summed in 32 bits; P and dS are rounded to the
 * tensors' type before their products (as q, k and v are; in fp16, which small
 * gradients would leave, as a power of two times them that follows d_o's size); maxima,
 * sums of exponentials, D and lse are in 32 bits.  Results repeat bit for bit: nothing is
 * added in an order that timing decides.
 *
 * Heads.  Element (b, s, h, e) of a tensor is data[b * stride_batch + s * stride_seq
 * + h * stride_head + e], so the head-sharded buffers that basp_seq2head writes (a
 * rank's sequences are the batch), packed projections and sequence-first orders are
 * all read in place.  `data` is 16-byte aligned and strides are multiples of 8
 * elements.  An input's stride may be 0.
 *
 * Conventions as in basp_fp8.h: the caller owns every buffer, nothing is allocated,
 * nothing synchronises, arguments are checked before anything is enqueued on
 * `stream`, offsets are 64 bits wide.  Outputs may not overlap any other buffer.
 */
#ifndef BASP_ATTENTION_H
#define BASP_ATTENTION_H

#include "basp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct basp_attention_desc {
    int64_t batch, q_len, k_len;   /* sequences (below 2^31), Sq, Sk (2^31 - 2^12)    */
    int64_t q_heads, k_heads;      /* Hq, Hkv: Hq a multiple of Hkv                   */
    int64_t head_dim;              /* a multiple of 8, 8 to 128                       */
    int64_t window;                /* keys a query sees with its own, >= 1; 0: all    */
    int64_t sinks;                 /* first keys that stay visible, >= 0              */
    float scale;                   /* finite, of the products q . k                   */
    basp_dtype dtype;              /* BF16 or FP16, of every tensor                   */
} basp_attention_desc;

typedef struct basp_heads {
    void *data;
    int64_t stride_batch, stride_seq, stride_head;   /* in elements, >= 0 */
} basp_heads;

/*
 * o [batch][Sq][Hq][d] from q (the same), k and v [batch][Sk][Hkv][d].
 *   o_rest   as o, of 8-bit integers, 8-byte aligned: what o lost when it was rounded, in
 *            256ths of its last place, or NULL.  The backward's D is then made of both,
 *            which matters where a query sees few keys
 *   lse      [batch][Hq][Sq] fp32 (the backward takes it), or NULL
 */
basp_status basp_attention(const basp_attention_desc *desc, const basp_heads *q, const basp_heads *k,
                           const basp_heads *v, const basp_heads *o, const basp_heads *o_rest, float *lse,
                           cudaStream_t stream);

/*
 * Gradients.  o, o_rest (or NULL) and lse as basp_attention wrote them.
 *   workspace   device scratch of basp_attention_backward_workspace(desc) bytes,
 *               16-byte aligned
 */
basp_status basp_attention_backward(const basp_attention_desc *desc, const basp_heads *q, const basp_heads *k,
                                    const basp_heads *v, const basp_heads *o, const basp_heads *o_rest,
                                    const float *lse, const basp_heads *d_o, const basp_heads *dq, const basp_heads *dk,
                                    const basp_heads *dv, void *workspace, size_t workspace_bytes,
                                    cudaStream_t stream);
int64_t basp_attention_backward_workspace(const basp_attention_desc *desc);

/*
 * One new token of each sequence over a cache (q_len = 1; k_len is the cache's
 * capacity).  Sequence b holds lengths[b] tokens, the new one, whose key and value
 * are in the cache already, the last of them: it sees key j if j < lengths[b] and
 * (j >= lengths[b] - window or j < sinks).  Nothing else of the cache is read.
 *   lengths     [batch] in device memory, read when the kernel runs (so a captured
 *               call can be replayed); below 0 counts as 0, above k_len as k_len.
 *               A sequence of no tokens has o = 0.
 *   workspace   device scratch of basp_attention_decode_workspace(desc) bytes, 16-byte
 *               aligned; may be NULL where that is 0
 */
basp_status basp_attention_decode(const basp_attention_desc *desc, const basp_heads *q, const basp_heads *k,
                                  const basp_heads *v, const int32_t *lengths, const basp_heads *o,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream);
int64_t basp_attention_decode_workspace(const basp_attention_desc *desc);

/*
 * The kernels wait for their own asynchronous copies and matrix instructions, each
 * wait with a limit far above what any wait takes.  A wait that runs out ends the
 * kernel in order, leaves NaN in what it was computing, and is counted.  This call
 * reads and clears the count on the current device; it synchronises the device.
 * Zero in any healthy run.
 */
basp_status basp_attention_timeouts(unsigned long long *count);

#ifdef __cplusplus
}
#endif

#endif /* BASP_ATTENTION_H */
