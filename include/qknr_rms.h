/*
 * qknr_rms.h — C ABI of the root-mean-square norm of token rows, with the
 * residual's addition before it, an output in 8 bits with scales, and its
 * backward pass, in libqknr.so.
 *
 * x is [T, C] rows of the activation dtype, residual (optional) likewise.
 * Row t belongs to sample b = t / rows_per_batch and takes weight row b; its
 * gain is weight, 1 + weight with QKNR_RMS_UNIT_OFFSET (a modulation), or 1
 * without a weight.  Per row, over its C values,
 *
 *     h    = x + residual               sum  = h rounded to the activation dtype
 *     rstd = rsqrt(mean_c(h^2) + eps)
 *     y    = h * rstd * gain
 *
 * (the norm sees the sum before its rounding).  With out = QKNR_RMS_OUT_E4M3
 * y holds 8-bit floats (e4m3, no infinities) and scales the fp32 factors that
 * take them back, one per row (scale_block 0) or one per 128 columns:
 *
 *     scale = max(max|h * rstd * gain| / 448, 2^-126)      y = h * rstd * gain * (1 / scale)
 *
 * with the reciprocal rounded to fp32 (a value next to the middle of two 8-bit
 * ones may go to the other one than the quotient would); a NaN in the values a scale covers makes all of them, and the scale, NaN.
 *
 * The backward pass takes x = h as the forward pass rounded it (its sum, or x
 * where there was no residual), its rstd, dy = dL/dy and, optionally, dsum,
 * the gradient that reaches h past the norm.  With xhat = x * rstd and
 * g = dy * gain,
 *
 *     dx[c]        = rstd * (g[c] - xhat[c] * mean_c(g * xhat)) + dsum[c]
 *     dweight[b,c] = sum over the rows t of b of dy[t, c] * xhat[t, c]
 *
 * dx is the gradient of the forward pass's x and of its residual alike.
 *
 * Everything is computed in fp32 and rounded once, to nearest even; dweight
 * stays fp32 and is summed in a fixed order (no atomics), so equal calls give
 * equal bits.
 *
 * Ownership and errors follow qknr.h: the caller owns every buffer (the
 * backward pass's workspace included), the library allocates nothing and
 * never synchronises; argument errors return before any CUDA call; a bounded
 * in-kernel wait that runs out writes QKNR_ERR_TIMEOUT to *dev_status.
 */
#ifndef QKNR_RMS_H_
#define QKNR_RMS_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QKNR_RMS_UNIT_OFFSET 0x10u  /* flags: the gain is 1 + weight */

#define QKNR_RMS_OUT_SAME 0         /* y in the activation dtype */
#define QKNR_RMS_OUT_E4M3 1         /* y in 8 bits, with scales */

typedef struct qknr_rms_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* x, residual, sum and the gradients: QKNR_BF16 or QKNR_FP16 */
  const void *x;              /* device [T, C] */
  const void *residual;       /* device [T, C], or NULL */
  void *sum;                  /* device [T, C]; required with a residual; may be it, or x (same stride) */
  void *y;                    /* device [T, C]; may be x in the activation dtype (same stride) */
  int64_t x_stride, residual_stride, sum_stride, y_stride;   /* elements per row; 0 = C */
  int64_t tokens;             /* T */
  int32_t hidden;             /* C: a multiple of 8 (scale_block 128: of 128), at most 32768 */
  int64_t rows_per_batch;     /* rows sharing one weight row; 0 = all of them */
  const void *weight;         /* device [B, C], B = ceil(T / rows_per_batch); may be NULL */
  int32_t param_dtype;        /* weight: QKNR_FP32, or the activation dtype */
  int64_t param_stride;       /* elements between weight rows; 0 = C */
  float eps;                  /* default 1e-6 (forward) */
  float *rstd;                /* device [T]; forward: written where not NULL; backward: required */
  int32_t out;                /* QKNR_RMS_OUT_SAME or QKNR_RMS_OUT_E4M3 */
  int32_t scale_block;        /* E4M3: 0 = a scale per row, 128 = a scale per 128 columns */
  float *scales;              /* E4M3: device [T] or [T, C / 128] */
  /* backward only */
  const void *dy;             /* device [T, C] */
  const void *dsum;           /* device [T, C], or NULL */
  void *dx;                   /* device [T, C]; may be dy or dsum (same stride) */
  int64_t dy_stride, dsum_stride, dx_stride;   /* elements per row; 0 = C */
  float *dweight;             /* device [B, C], contiguous; may be NULL */
  void *workspace;            /* device, 16-byte aligned, qknr_rms_workspace_bytes */
  size_t workspace_bytes;
  int32_t *dev_status;        /* optional device int32 (see qknr.h) */
  uint32_t flags;             /* QKNR_FLAG_NO_OVERLAP, QKNR_FLAG_TEST_STALL, QKNR_RMS_UNIT_OFFSET */
  uint64_t wait_limit_ns;     /* 0 = 2 s */
} qknr_rms_args;

/* Defaults: bf16, fp32 weight, eps 1e-6, an output in the activation dtype,
   everything else zero. */
void qknr_rms_args_init(qknr_rms_args *a);

/* Validate and launch the forward pass on `stream` (asynchronous, one
   kernel).  Base addresses and row strides must be 16-byte aligned (an 8-bit
   y: 8-byte; rstd and scales: 4-byte).  Outputs must not share an element
   with each other, nor with an input but as said above. */
qknr_status qknr_rms_forward(const qknr_rms_args *args, qknr_stream_t stream);

/* Device bytes qknr_rms_backward needs at `workspace` for these arguments
   (pointers are not looked at). */
qknr_status qknr_rms_workspace_bytes(const qknr_rms_args *args, size_t *bytes);

/* Validate and launch the backward pass on `stream` (asynchronous): one
   kernel that writes dx and partial sums of dweight, and one that adds the
   partial sums; rows of more than 8192 values take a third that sums each row
   first. */
qknr_status qknr_rms_backward(const qknr_rms_args *args, qknr_stream_t stream);

/* sizeof(qknr_rms_args) as compiled into the library. */
size_t qknr_rms_sizeof_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_RMS_H_ */
