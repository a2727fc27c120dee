/*
 * basp_optim.h -- C ABI of the optimiser's step over many tensors (same library,
 * libbasp.so, and same conventions as basp.h and basp_fp8.h).
 *
 * basp_adamw takes one step of Adam with decoupled weight decay (Loshchilov and
 * Hutter, "Decoupled Weight Decay Regularization", 2019).  For each element, with
 * t the step's number, counted from 1:
 *     m' = beta1 m + (1 - beta1) g          v' = beta2 v + (1 - beta2) g^2
 *     p' = p (1 - lr weight_decay)
 *          - lr / (1 - beta1^t) * m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
 * in 32 bits; p' is rounded once to its type.
 *
 * States in 8 bits.  m and the root of v are held in e4m3, with one power-of-two
 * scale (e8m0) for each 128 elements of a tensor: the least 2^e with
 * amax <= 448 * 2^e, as in basp_fp8.h.  The root has half of v's exponent range,
 * which 8 bits can hold; a root that is not zero is not rounded to zero.  The step
 * itself uses m' and v' before they are rounded.  They are rounded at random, up
 * with the fraction's probability: rounded to nearest, a state would never move by
 * the 0.1 % a step that beta2 = 0.999 asks for.
 *
 * The random bits are a function of the seed, the step, the tensor's place in the
 * list and the element's place in the tensor:
 *     mix(x):  x ^= x >> 16; x *= 0x6A09E667; x ^= x >> 15; x *= 0xBB67AE85; x ^= x >> 16
 *     key = mix(mix(mix(seed) ^ t) ^ tensor)
 *     bits = mix(i * 0x9E3779B9 + key)        (all modulo 2^32)
 * the low 16 for m and the high 16 for the root; a magnitude of k + f steps of the
 * e4m3 grid becomes k + 1 if f + (r + 1/2) / 2^16 >= 1, else k.  The constants are
 * the first 32 bits of the fractions of the golden ratio and of the roots of 2 and 3.
 */
#ifndef BASP_OPTIM_H
#define BASP_OPTIM_H

#include "basp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One tensor of n elements, in device memory, each buffer dense.  Buffers of one
 * call may not overlap (between tensors, of which there may be thousands, only p is
 * checked: no parameter may come twice). */
typedef struct basp_adamw_tensor {
    void *p;               /* n of `dtype` (BF16, FP16 or FP32): updated          */
    const void *g;         /* n of `grad_dtype`: `dtype` or FP32                  */
    void *m, *v;           /* n fp32 each, or n e4m3 each (m and the root of v)   */
    void *m_scales, *v_scales;   /* ceil(n / 128) e8m0 each; NULL: 32-bit states  */
    int64_t n;
    basp_dtype dtype, grad_dtype;
} basp_adamw_tensor;

typedef struct basp_adamw_options {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;          /* t, from 1 to 2^31 - 1; not used with step_at         */
    const int32_t *step_at;/* device memory: t is read when the kernel runs, so that
                              a captured call can be replayed; or NULL             */
    uint32_t seed;         /* of the 8-bit states' rounding                        */
} basp_adamw_options;

/*
 * One step over `count` tensors, in one launch for each few hundred of them.  All
 * tensors have 32-bit states or all have 8-bit states.  A tensor of no elements is
 * valid.  Arguments are checked before anything is enqueued on `stream`; the tables
 * are copied before the call returns.
 */
basp_status basp_adamw(const basp_adamw_tensor *tensors, int64_t count,
                       const basp_adamw_options *options, cudaStream_t stream);

/*
 * The same for tensors that have taken different numbers of steps, or that come in
 * other lists from step to step.  Both in host memory:
 *   steps_at    [count]: for each tensor where its own t is in device memory, read as
 *               step_at is; the options' step and step_at are not used.  Or NULL
 *   numbers     [count]: the tensors' numbers for the random bits, in place of their
 *               places in the list; or NULL
 */
basp_status basp_adamw_each(const basp_adamw_tensor *tensors, const int32_t *const *steps_at, const uint32_t *numbers,
                            int64_t count, const basp_adamw_options *options, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BASP_OPTIM_H */
