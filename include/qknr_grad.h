/*
 * qknr_grad.h — C ABI of the backward pass of the fused QK-RMSNorm + RoPE
 * (qknr.h) in libqknr.so.
 *
 * With x a head's D inputs, r = rsqrt(sum_d x[d]^2 / D + eps) and do the
 * gradient of that head's outputs, per token and head:
 *
 *     dy[d] = do[d] * cos[d] + s(p(d)) * do[p(d)] * sin[p(d)]
 *     g[d]  = dy[d] * gamma[d]
 *     dx[d] = r * (g[d] - x[d] * r^2 * sum_d(g * x) / D)
 *     dgamma[d] = sum over tokens and heads of dy[d] * x[d] * r
 *
 * p(d) and s(d) are qknr.h's rotation partner and sign.  x is the input of
 * qknr_forward, so a caller who trains runs that out of place.  Everything
 * is computed in fp32; dx is rounded once, to nearest even, into the
 * activation dtype, dgamma_q and dgamma_k stay fp32, summed in a fixed order
 * (no atomics).  The V columns' gradient passes through: left alone, or
 * copied bit for bit.
 *
 * Layouts, table forms, ownership and errors are qknr.h's: the caller owns
 * every buffer (the workspace included), the library allocates nothing and
 * never synchronises.
 */
#ifndef QKNR_GRAD_H_
#define QKNR_GRAD_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qknr_grad_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* activations and their gradients: QKNR_BF16 or QKNR_FP16 */
  const void *q, *k;          /* device: the forward call's inputs */
  const void *dq, *dk, *dv;   /* device: gradients of its outputs */
  void *dq_out, *dk_out, *dv_out;   /* device: gradients of its inputs; NULL or dq / dk (same stride) = in place;
                                       dv is copied only when dv_out is non-NULL and differs from dv */
  int64_t q_stride, k_stride;                          /* elements per row; 0 = H*D */
  int64_t dq_stride, dk_stride, dv_stride;             /* 0 = H*D */
  int64_t dq_out_stride, dk_out_stride, dv_out_stride; /* 0 = the gradient's */
  int64_t tokens;             /* T; 0: no rows, dgamma_q and dgamma_k are zeroed */
  int32_t n_heads_q, n_heads_k, n_heads_v;
  int32_t head_dim;           /* D: 64 or 128 */
  const float *gamma_q, *gamma_k;   /* device fp32 [D] */
  float eps;                  /* the forward call's; default 1e-6 */
  const void *cos, *sin;      /* device tables, qknr_cos_layout */
  int32_t cos_dtype, cos_layout;
  int64_t cos_rows;           /* 0 = tokens.  Row of token t: t % cos_rows */
  int32_t rope_style;
  float *dgamma_q, *dgamma_k; /* device fp32 [D]; either may be NULL; not touched where its tensor has no heads */
  void *workspace;            /* device, 16-byte aligned, qknr_grad_workspace_bytes */
  size_t workspace_bytes;
  int32_t *dev_status;        /* optional device int32, written by checked builds only */
  uint32_t flags;             /* QKNR_FLAG_NO_OVERLAP */
} qknr_grad_args;

/* Defaults: bf16, fp32 shared cos/sin, interleaved, eps 1e-6. */
void qknr_grad_args_init(qknr_grad_args *a);

/* Device bytes qknr_backward needs at `workspace` (pointers are not looked at). */
qknr_status qknr_grad_workspace_bytes(const qknr_grad_args *args, size_t *bytes);

/* Validate and launch on `stream` (asynchronous): one kernel that writes the
   gradients and partial sums of dgamma, and one that adds those.  Base
   addresses and row strides must be 16-byte aligned.  A gradient output may
   be its own incoming gradient; it must not otherwise share an element
   with an input or another output (columns of one buffer may interleave). */
qknr_status qknr_backward(const qknr_grad_args *args, qknr_stream_t stream);

/* sizeof(qknr_grad_args) as compiled into the library. */
size_t qknr_sizeof_grad_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_GRAD_H_ */
