/*
 * swiglu_norm.h -- C ABI of libswiglu, part four: the layer norm in front of
 * linear_fc1, forward and backward.
 *
 * Conventions of swiglu.h: device pointers owned by the caller, sizes and
 * strides in elements, every argument checked on the host before anything is
 * launched, work enqueued on `stream`, nothing allocated, capturable into a
 * CUDA graph, status codes of swiglu.h.
 *
 * For every row of x [rows, n]:
 *   mean = sum_j x / n,  rstd = 1 / sqrt(sum_j (x - mean)^2 / n + eps)
 *   xhat = (x - mean) rstd,  y = xhat * w + b
 * x, y, dy and dx are of `dtype`; w and b, [n], and their gradients are of
 * `param_dtype`: `dtype` or SWIGLU_F32.  mean and rstd are fp32.  Arithmetic
 * is fp32; each result is rounded once.  A NaN or an infinity in a row makes
 * that row NaN and no other.
 */
#ifndef LIBSWIGLU_SWIGLU_NORM_H
#define LIBSWIGLU_SWIGLU_NORM_H

#include "swiglu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of rows of a call (n: SWIGLU_MAX_N). */
#define SWIGLU_NORM_MAX_ROWS 2147483647

/*
 * y (and, where not NULL, mean and rstd, [rows] each) from x, w and b; w and b may
 * be NULL (ones, zeros).  Row strides of x and y >= n; eps >= 0 and finite (else
 * SWIGLU_ERR_SHAPE).  Outputs overlap nothing (SWIGLU_ERR_ALIAS).
 */
swiglu_status_t swiglu_layer_norm_fwd(const void *x, const void *w, const void *b, void *y,
                                      float *mean, float *rstd, int64_t rows, int64_t n,
                                      int64_t x_row_stride, int64_t y_row_stride, float eps,
                                      swiglu_dtype_t dtype, swiglu_dtype_t param_dtype,
                                      swiglu_stream_t stream);

/*
 * With h = dy w (dy without w):
 *   dx = rstd (h - mean_j(h) - xhat mean_j(h xhat))
 *   dw = sum over rows of dy xhat   (dw may be NULL)
 *   db = sum over rows of dy        (db may be NULL)
 * mean and rstd are those of the forward.  Row strides of dy, x and dx >= n.  The
 * column sums are fp32, in an order that depends on the sizes, the alignment and
 * the device alone: the same call gives the same bits.  (Rows are shared out among
 * chains of additions: 16 on each SM up to 512 columns, 8, 4 and 2 up to 1024, 2048 and
 * 4096, one up to 8192; two for each cluster of 4 CTAs, of 8 beyond 16384 columns, that
 * the device runs at a time, 38 and 19 of them at most.  Beyond 32768 columns, where chains may
 * be as few as one, they are cut into segments of 256 rows.  The segments and the chains of
 * an SM, then the SMs' sums in 16 chains, are added up in their order.)  They take a workspace of
 * swiglu_layer_norm_bwd_workspace_size(rows, n, dtype) bytes, 16-byte aligned
 * (else SWIGLU_ERR_WORKSPACE), which may be used again by work later in the
 * stream, and not by work that runs at the same time.  Outputs and workspace
 * overlap nothing (SWIGLU_ERR_ALIAS).  rows == 0: dw and db are set to
 * zero.
 */
swiglu_status_t swiglu_layer_norm_bwd_workspace_size(int64_t rows, int64_t n, swiglu_dtype_t dtype,
                                                     size_t *bytes);

swiglu_status_t swiglu_layer_norm_bwd(const void *dy, const void *x, const float *mean,
                                      const float *rstd, const void *w, void *dx, void *dw,
                                      void *db, void *workspace, size_t workspace_bytes,
                                      int64_t rows, int64_t n, int64_t dy_row_stride,
                                      int64_t x_row_stride, int64_t dx_row_stride,
                                      swiglu_dtype_t dtype, swiglu_dtype_t param_dtype,
                                      swiglu_stream_t stream);

/* *flag = 1 if any launch above gave up on an internal wait so far (its results are then
 * undefined), else 0.  Synchronises with the current device. */
swiglu_status_t swiglu_layer_norm_timeout_flag(int *flag);

#ifdef __cplusplus
}
#endif

#endif /* LIBSWIGLU_SWIGLU_NORM_H */
