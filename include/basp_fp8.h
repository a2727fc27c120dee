/*
 * basp_fp8.h -- C ABI of the 8-bit projections on both sides of the re-layout
 * (same library, libbasp.so, and same conventions as basp.h).
 *
 * A sequence-parallel attention layer norms the residual stream, projects it
 * to a packed QKV activation (the input of basp_seq2head_qkv), attends, and
 * projects the re-laid-out output (the result of basp_head2seq).  The calls
 * here do the norm and the two projections with 8-bit operands, forward and
 * backward:
 *   basp_rmsnorm            residual addition + root-mean-square norm, with an
 *                           8-bit output, a 16/32-bit output, or both
 *   basp_rmsnorm_backward   its gradient
 *   basp_quantize_fp8       a 16/32-bit matrix (and its transpose) to 8 bits
 *   basp_matmul_fp8         C = A B^T of two 8-bit matrices
 * The gradients of a projection Y = X W^T are two more products:
 * dX = dY W (rows of dY against the transpose of W) and dW = dY^T X (both
 * operands transposed, the tokens summed over).
 *
 * 8-bit matrices.  Values are e4m3 (4 exponent bits, 3 mantissa bits, largest
 * 448, no infinities).  A block of 1 x 128 or 128 x 128 values shares one
 * scale 2^e, stored as the byte e + 127 (e8m0).  The element stands for
 * value * 2^e.  Scales are powers of two because the tensor cores of sm_103a
 * apply exactly those inside the product, at no cost; the rounding error of
 * an e4m3 value is relative, so a finer scale would gain nothing but the
 * last bit of range.  The quantising calls take the least e for which the
 * block's largest finite magnitude is at most 448 * 2^e (a block of zeros:
 * e = 0; e is at least -127), round to nearest even, and store infinities
 * and NaN as NaN.
 *
 * Conventions as in basp.h: the caller owns every buffer, nothing is
 * allocated, nothing synchronises, arguments are checked before anything is
 * enqueued on `stream`, and kernels use programmatic dependent launch but
 * read and write nothing before the previous kernel on `stream` is done.
 * Row strides are in elements of the matrix's own type.  Offsets are 64 bits
 * wide; rows and columns are each below 2^31.  A matrix of zero rows or
 * columns is valid and launches nothing (a product over zero columns gives
 * the bias or zeros).  Outputs may not overlap inputs or each other, except
 * where a call says so: BASP_ERR_ALIASING.
 */
#ifndef BASP_FP8_H
#define BASP_FP8_H

#include "basp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values that share a scale along a row. */
#define BASP_FP8_BLOCK 128

/* An 8-bit matrix in device memory.  Row r of the values starts at
 * data + r * pitch; `pitch` is a multiple of 16 and `data` 16-byte aligned.
 * Scale (i, j) belongs to rows [i * block_rows, (i+1) * block_rows) and
 * columns [128 j, 128 (j+1)) and is the byte scales[i * scale_pitch + j];
 * `scale_pitch` is a multiple of 4 and `scales` 4-byte aligned.  Bytes
 * between the end of a row and its pitch are never used and never written. */
typedef struct basp_fp8_matrix {
    void *data;
    void *scales;
    int64_t rows, cols;
    int64_t pitch;         /* >= cols, % 16 == 0            */
    int64_t scale_pitch;   /* >= ceil(cols / 128), % 4 == 0 */
    int64_t block_rows;    /* 1 or 128                      */
} basp_fp8_matrix;

/*
 * h = x + residual (rounded to `dtype`; h = x without a residual),
 * rstd = (mean(h^2) + eps)^-1/2 over each row, y = h * rstd * weight.
 * Sums are in 32 bits; h * rstd and its product with the weight are rounded to
 * 32 bits each, and y once, to `dtype` or to 8 bits.  Results repeat bit for bit;
 * the order of a row's sum, and so the last bit of rstd, depends on the number of
 * rows and columns and on their alignment.
 *   x, residual   [rows][cols] of `dtype` (BF16, FP16 or FP32); residual may
 *                 be NULL
 *   weight        [cols] of `weight_dtype`: `dtype` or FP32
 *   h             [rows][cols] of `dtype`, or NULL; may be the very buffer of
 *                 x or residual (same address and stride)
 *   y             [rows][cols] of `dtype`, or NULL
 *   q             8-bit y (rows x cols, block_rows = 1), or NULL
 *   rstd          [rows] fp32, or NULL (rows without columns: not written)
 * At least one of y and q is given.
 */
basp_status basp_rmsnorm(basp_dtype dtype, int64_t rows, int64_t cols,
                         const void *x, int64_t x_stride,
                         const void *residual, int64_t residual_stride,
                         const void *weight, basp_dtype weight_dtype, float eps,
                         void *h, int64_t h_stride, void *y, int64_t y_stride,
                         const basp_fp8_matrix *q, float *rstd, cudaStream_t stream);

/*
 * Gradient of basp_rmsnorm (the rounding of y is passed through):
 *   g = dy * weight, n = h * rstd,
 *   dx = rstd * (g - n * mean(g * n)) + dh, which is the gradient of x and of
 *        the residual alike;
 *   dweight = sum over rows of dy * n.
 *   dy            [rows][cols] of `dtype`
 *   h, rstd       as basp_rmsnorm wrote them (h = x without a residual)
 *   dh            [rows][cols] of `dtype`: the gradient that reaches h past
 *                 the norm; or NULL
 *   dx            [rows][cols] of `dtype`; may be the very buffer of dy or dh
 *   dweight       [cols] fp32, or NULL
 *   workspace     device scratch of basp_rmsnorm_backward_workspace(rows,
 *                 cols) bytes (16-byte aligned); may be NULL without dweight
 * The rows are summed in an order that the sizes alone fix, so results repeat
 * bit for bit.
 */
basp_status basp_rmsnorm_backward(basp_dtype dtype, int64_t rows, int64_t cols,
                                  const void *dy, int64_t dy_stride,
                                  const void *h, int64_t h_stride, const float *rstd,
                                  const void *weight, basp_dtype weight_dtype,
                                  const void *dh, int64_t dh_stride,
                                  void *dx, int64_t dx_stride, float *dweight,
                                  void *workspace, size_t workspace_bytes,
                                  cudaStream_t stream);

/* Workspace of basp_rmsnorm_backward with dweight, in bytes.  Host only. */
int64_t basp_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * x [rows][cols] of `dtype` -> 8 bits.
 *   q             rows x cols, or NULL
 *   qt            the transpose: cols x rows, with scales of its own along
 *                 its rows (the rows of x), or NULL
 * At least one is given; where both are, they have the same block_rows.  With
 * block_rows = 128 the two hold the same values and scales, transposed.
 */
basp_status basp_quantize_fp8(basp_dtype dtype, int64_t rows, int64_t cols,
                              const void *x, int64_t x_stride,
                              const basp_fp8_matrix *q, const basp_fp8_matrix *qt,
                              cudaStream_t stream);

/*
 * C [a->rows][b->rows] = A B^T (+ bias) (+ C): for 8-bit A (M x K) and
 * B (N x K), products summed in 32 bits and rounded once.
 *   bias          [N] of `dtype`, added to every row; or NULL
 *   accumulate    nonzero: add to what C holds (gradients over micro-batches)
 *   c             [M][N] of `dtype` (BF16, FP16 or FP32)
 * Results repeat bit for bit: where the sum over K is split, its parts are
 * joined in a fixed order.
 */
basp_status basp_matmul_fp8(const basp_fp8_matrix *a, const basp_fp8_matrix *b,
                            const void *bias, int accumulate, basp_dtype dtype,
                            void *c, int64_t c_stride, cudaStream_t stream);

/*
 * The product's kernel waits for its own asynchronous copies and matrix
 * instructions, each wait with a limit far above what any wait takes.  A
 * wait that runs out ends the kernel in order, leaves NaN in the part of C it
 * was computing, and is counted.  This call reads and clears the count on the
 * current device; it synchronises the device.  Zero in any healthy run.
 */
basp_status basp_matmul_fp8_timeouts(unsigned long long *count);

#ifdef __cplusplus
}
#endif

#endif /* BASP_FP8_H */
