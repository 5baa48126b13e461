/*
 * qknr_ln.h — C ABI of layer norm with its backward pass in libqknr.so, in
 * the plain affine form and in the modulated form of qknr_adaln.h.
 *
 * For every token row t of x [T, C], with parameter row b = t /
 * rows_per_batch (one row for all where rows_per_batch is 0) and
 *
 *     gain[c] = weight[b, c]       (QKNR_LN_UNIT_OFFSET: 1 + weight[b, c];
 *                                   1 where weight is NULL)
 *
 * the forward pass writes
 *
 *     mean = sum_c x[c] / C,   var = sum_c (x[c] - mean)^2 / C
 *     rstd = 1 / sqrt(var + eps)
 *     y[c] = (x[c] - mean) * rstd * gain[c] + bias[b, c]
 *
 * and, where asked for, mean and rstd of each row in fp32.  The backward
 * pass takes dy = dL/dy and those two, and with xhat = (x - mean) * rstd and
 * g[c] = dy[c] * gain[c] writes
 *
 *     dx[c]        = rstd * (g[c] - mean_c(g) - xhat[c] * mean_c(g * xhat))
 *     dweight[b,c] = sum over the rows t of b of dy[t, c] * xhat[t, c]
 *     dbias[b,c]   = sum over the rows t of b of dy[t, c]
 *
 * Everything is computed in fp32; y and dx are rounded once, to nearest
 * even, into the activation dtype, dweight and dbias stay fp32.  The sums
 * over rows are taken in a fixed order (no atomics), so equal calls give
 * equal bits.
 *
 * Ownership and errors follow qknr.h: the caller owns every buffer
 * (the backward pass's workspace included), the library allocates nothing
 * and never synchronises; argument errors return before any CUDA call; a
 * bounded in-kernel wait that runs out writes QKNR_ERR_TIMEOUT to
 * *dev_status.
 */
#ifndef QKNR_LN_H_
#define QKNR_LN_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QKNR_LN_UNIT_OFFSET 0x10u   /* flags: the gain is 1 + weight */

typedef struct qknr_ln_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* x, y, dy and dx: QKNR_BF16 or QKNR_FP16 */
  const void *x;              /* device [T, C], row stride x_stride elements */
  void *y;                    /* forward: device [T, C]; NULL or x (same stride) = in place */
  int64_t x_stride, y_stride; /* elements per row; 0 = C (y: x's) */
  int64_t tokens;             /* T; 0: no rows, dweight and dbias are zeroed where rows_per_batch is 0 */
  int32_t hidden;             /* C: a multiple of 8, at most 32768 */
  int64_t rows_per_batch;     /* rows sharing one parameter row; 0 = all of them */
  const void *weight, *bias;  /* device [B, C], B = ceil(T / rows_per_batch); either may be NULL */
  int32_t param_dtype;        /* weight and bias: QKNR_FP32, or the activation dtype */
  int64_t param_stride;       /* elements between parameter rows; 0 = C */
  float eps;                  /* default 1e-6 (forward) */
  float *mean, *rstd;         /* device [T]; forward: written where not NULL; backward: required */
  /* backward only */
  const void *dy;             /* device [T, C] */
  void *dx;                   /* device [T, C]; NULL or dy (same stride) = in place of dy */
  int64_t dy_stride, dx_stride;   /* elements per row; 0 = C (dx: dy's) */
  float *dweight, *dbias;     /* device [B, C], contiguous; either may be NULL */
  void *workspace;            /* device, 16-byte aligned, qknr_ln_workspace_bytes */
  size_t workspace_bytes;
  int32_t *dev_status;        /* optional device int32 (see qknr.h) */
  uint32_t flags;             /* QKNR_FLAG_NO_OVERLAP, QKNR_FLAG_TEST_STALL, QKNR_LN_UNIT_OFFSET */
  uint64_t wait_limit_ns;     /* 0 = 2 s */
} qknr_ln_args;

/* Defaults: bf16, fp32 parameters, eps 1e-6, everything else zero. */
void qknr_ln_args_init(qknr_ln_args *a);

/* Validate and launch the forward pass on `stream` (asynchronous, one
   kernel).  Base addresses and row strides must be 16-byte aligned (mean
   and rstd: 4-byte); `y` must not share an element with an input
   unless it is x, mean and rstd none with any other tensor. */
qknr_status qknr_ln_forward(const qknr_ln_args *args, qknr_stream_t stream);

/* Device bytes qknr_ln_backward needs at `workspace` for these arguments
   (pointers are not looked at). */
qknr_status qknr_ln_workspace_bytes(const qknr_ln_args *args, size_t *bytes);

/* Validate and launch the backward pass on `stream` (asynchronous): one
   kernel that writes dx and partial sums of dweight and dbias, and one that
   adds the partial sums; rows of more than 8192 values take a third that
   sums each row first.  dx may be dy; outputs must not otherwise share
   an element with an input (columns of one buffer may interleave). */
qknr_status qknr_ln_backward(const qknr_ln_args *args, qknr_stream_t stream);

/* sizeof(qknr_ln_args) as compiled into the library. */
size_t qknr_ln_sizeof_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_LN_H_ */
