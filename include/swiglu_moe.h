/*
 * swiglu_moe.h -- C ABI of libswiglu, part two: the routed experts' MLP.
 *
 * Two sets of operators around the SwiGLU of swiglu.h (same conventions: device
 * pointers owned by the caller, sizes and strides in elements, every argument
 * checked on the host before anything is launched, work enqueued on `stream`,
 * nothing allocated, capturable into a CUDA graph, status codes of swiglu.h):
 *
 *   - the experts' matrix products, one weight matrix per expert, over rows
 *     sorted by expert (ragged groups), forward and both gradients, with the
 *     activation fused into the first of them;
 *   - the activation that keeps its input in 8 bits for the backward pass
 *     (the counterpart of Megatron's fp8_input_store), and that backward pass.
 *
 * GROUPS.  Rows 0 .. rows - 1 are sorted by expert.  `ends` is a DEVICE vector
 * of `groups` int32: group e holds rows [start_e, end_e) with
 *   start_e = max(0, ends[0], ..., ends[e - 1]),  end_e = max(start_e, ends[e]),
 * both at most `rows`: the running sum of the rows per expert, of which any
 * value is safe.  A group may be empty.  Rows from the last end on belong to
 * no group: their outputs are zero, and they enter no weight gradient.  The
 * host never reads `ends`, so the groups may change between replays of a
 * captured graph.
 *
 * 8-BIT CHECKPOINT of a tensor x [rows, 2n] (gate columns [0, n), up columns
 * [n, 2n)).  Each half of a row is cut into nb = ceil(n / 32) blocks of 32
 * columns (the last one may be shorter).  A block stores one code per element
 * and one scale:
 *   scales [rows, 2 nb] bytes, the gate half's blocks first: c stands for
 *          2^(c - 127); c is the smallest value >= 0 for which every finite |x|
 *          of the block is at most 448 * 2^(c - 127)   (E8M0; 255 is not used)
 *   q      [rows, 2n] bytes: x * 2^(127 - c) rounded to nearest even to e4m3
 *          (4 significant bits, largest value 448); infinities and NaN become
 *          NaN.  Under the largest scale (c = 247) values above 240 keep the
 *          code of 240: 256 * 2^120 would be beyond fp32.
 * A power of two loses nothing by itself: an element within 2^-14 of its
 * block's largest keeps 4 significant bits (a relative error of at most 2^-4).
 */
#ifndef LIBSWIGLU_SWIGLU_MOE_H
#define LIBSWIGLU_SWIGLU_MOE_H

#include "swiglu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Columns per checkpoint block. */
#define SWIGLU_CKPT8_BLOCK 32

/* Largest number of groups of one call. */
#define SWIGLU_MAX_GROUPS 1024

/* Limits of the products' sizes (below; far beyond any memory but for the rows of
 * a weight gradient, which must be summed within the 2 s of an internal wait). */
#define SWIGLU_GROUPED_MAX_ROWS 2147483391
#define SWIGLU_GROUPED_MAX_ROWS_WGRAD 268435456
#define SWIGLU_GROUPED_MAX_FEATURES 1073741823

/*
 * Forward with an 8-bit checkpoint:
 *   y[r, j] = w[r] * silu(x[r, j]) * x[r, n + j]   (w NULL: no weights)
 *   q, scales = the checkpoint of x (above)
 *   x [rows, 2n] of `dtype`, y [rows, n] of `dtype`, w [rows] fp32 or NULL
 *   row strides: x >= 2n, y >= n, q >= 2n, scales >= 2 nb
 * y is that of swiglu_gateup_fwd / swiglu_gateup_weighted_fwd on x itself (not
 * on its checkpoint).  y, q and scales overlap nothing (SWIGLU_ERR_ALIAS).
 */
swiglu_status_t swiglu_ckpt8_fwd(const void *x, const float *w, void *y, void *q, void *scales,
                                 int64_t rows, int64_t n, int64_t x_row_stride,
                                 int64_t y_row_stride, int64_t q_row_stride,
                                 int64_t scale_row_stride, swiglu_dtype_t dtype,
                                 swiglu_stream_t stream);

/*
 * Backward from the checkpoint.  With g, u the values that q and scales stand
 * for, s = sigmoid(g) and d = w[r] * dy[r, j] (d = dy without weights):
 *   dx[r, j]     = d * u * s * (1 + g * (1 - s))
 *   dx[r, n + j] = d * g * s
 *   dw[r]        = sum_j dy[r, j] * silu(g) * u   (fp32, fixed order)
 *   y[r, j]      = w[r] * silu(g) * u             (when y is not NULL: the second
 *                  product's weight gradient needs it, so it need not be kept)
 *   dy [rows, n], dx [rows, 2n], y [rows, n] of `dtype`; w and dw [rows] fp32,
 *   both given or both NULL (SWIGLU_ERR_NULL).
 * dx, dw and y overlap nothing (SWIGLU_ERR_ALIAS).  With n == 0 the call sets
 * dw to zero.
 */
swiglu_status_t swiglu_ckpt8_bwd(const void *dy, const void *q, const void *scales, const float *w,
                                 void *dx, float *dw, void *y, int64_t rows, int64_t n,
                                 int64_t dy_row_stride, int64_t q_row_stride,
                                 int64_t scale_row_stride, int64_t dx_row_stride,
                                 int64_t y_row_stride, swiglu_dtype_t dtype,
                                 swiglu_stream_t stream);

/*
 * The experts' products (bf16 only, fp32 accumulation on the tensor cores,
 * every result rounded once; contiguous tensors, 16-byte aligned pointers).
 * The tensor cores truncate the running sum every 16 terms: a sum of D terms is
 * within D 2^-27 of the sum of their absolute values.  D is the depth of a
 * product over rows; weight gradients add up sums of at most 512 (fp32 dW) or
 * 131,072 rows (bf16 dW) with rounded fp32 additions.
 * For each row t of group e:
 *
 *   swiglu_grouped_mm_fwd     y[t, :]  = W[e] x[t, :]
 *     x [rows, K], W [groups, N, K], y [rows, N]
 *   swiglu_grouped_mm_dgrad   dx[t, :] = W[e]^T dy[t, :]
 *     dy [rows, N], W [groups, N, K], dx [rows, K]
 *   swiglu_grouped_mm_wgrad   dW[e]    = sum_{t in e} dy[t, :]^T x[t, :]
 *     dy [rows, N], x [rows, K], dW [groups, N, K] of dw_dtype (SWIGLU_BF16 or
 *     SWIGLU_F32); accumulate != 0 (SWIGLU_F32 only, else SWIGLU_ERR_DTYPE):
 *     dW[e] += the sum.  An empty group gives zeros (or leaves dW[e] as it is).
 *   swiglu_grouped_fc1_fwd    y[t, j]  = probs[t] * silu(g) * u,
 *       g = W[e][j] . x[t],  u = W[e][n + j] . x[t]
 *     x [rows, K], W [groups, 2n, K] (gate rows first), probs [rows] fp32 or
 *     NULL, y [rows, n]; the activation is applied to the fp32 accumulators.
 *     What the backward pass keeps, at most one of (both: SWIGLU_ERR_ALIAS):
 *       fc1 [rows, 2n] bf16 (g and u, rounded), or
 *       q [rows, 2n] and scales [rows, 2 nb], the checkpoint of the unrounded
 *       g and u (both given or both NULL).
 *
 * Requirements: N (n) and K multiples of 8 and at least 8, rows at most
 * SWIGLU_GROUPED_MAX_ROWS (dW: SWIGLU_GROUPED_MAX_ROWS_WGRAD), K and
 * groups * N at most SWIGLU_GROUPED_MAX_FEATURES, groups * 2n as well,
 * 1 <= groups <= SWIGLU_MAX_GROUPS, fewer than 2^29 tiles of 256 x 256 in a
 * result (else SWIGLU_ERR_SHAPE); pointers 16-byte aligned, ends and probs 4-byte aligned
 * (else SWIGLU_ERR_STRIDE); outputs overlap nothing (SWIGLU_ERR_ALIAS).  No row
 * reads another group's rows, so a NaN in one row reaches no other row's
 * outputs and no other group's dW.  rows == 0 is an empty call (wgrad: every
 * group is empty).  Sums are formed in an order that depends on the sizes and
 * the groups alone: the same call gives the same bits.
 */
swiglu_status_t swiglu_grouped_fc1_fwd(const void *x, const void *w, const int32_t *ends,
                                       const float *probs, void *y, void *fc1, void *q,
                                       void *scales, int64_t rows, int64_t groups, int64_t n,
                                       int64_t K, swiglu_dtype_t dtype, swiglu_stream_t stream);

swiglu_status_t swiglu_grouped_mm_fwd(const void *x, const void *w, const int32_t *ends, void *y,
                                      int64_t rows, int64_t groups, int64_t N, int64_t K,
                                      swiglu_dtype_t dtype, swiglu_stream_t stream);

swiglu_status_t swiglu_grouped_mm_dgrad(const void *dy, const void *w, const int32_t *ends,
                                        void *dx, int64_t rows, int64_t groups, int64_t N,
                                        int64_t K, swiglu_dtype_t dtype, swiglu_stream_t stream);

swiglu_status_t swiglu_grouped_mm_wgrad(const void *dy, const void *x, const int32_t *ends,
                                        void *dw, int64_t rows, int64_t groups, int64_t N,
                                        int64_t K, swiglu_dtype_t dtype, swiglu_dtype_t dw_dtype,
                                        int accumulate, swiglu_stream_t stream);

/* How a product of these sizes is computed (host only): *slices = 0, a pair of CTAs per
 * tile of 256 x 256; 1, 2, 4 or 8, that many CTAs, each a slice of the contraction, per
 * tile of 128 by at most 128.  N, K (fc1: n, K) and dw_dtype (read for the weight
 * gradient) as in the call itself; the choice follows from the sizes alone, and sums are
 * added in another order with another number of slices.  rows == 0: 0. */
typedef enum {
    SWIGLU_GROUPED_FC1 = 0,
    SWIGLU_GROUPED_MM = 1,
    SWIGLU_GROUPED_DGRAD = 2,
    SWIGLU_GROUPED_WGRAD = 3
} swiglu_grouped_product_t;

swiglu_status_t swiglu_grouped_slices(swiglu_grouped_product_t product, int64_t rows,
                                      int64_t groups, int64_t N, int64_t K,
                                      swiglu_dtype_t dw_dtype, int *slices);

/* *flag = 1 if any launch of the products above gave up on an internal wait so
 * far (its results are then undefined), else 0.  Synchronises with the current
 * device. */
swiglu_status_t swiglu_grouped_timeout_flag(int *flag);

#ifdef __cplusplus
}
#endif

#endif /* LIBSWIGLU_SWIGLU_MOE_H */
