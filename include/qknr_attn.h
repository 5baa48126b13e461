/*
 * qknr_attn.h — C ABI of attention and its backward pass in libqknr.so: the
 * step that the fused QK-RMSNorm + RoPE (qknr.h) prepares Q and K for.
 *
 * q is [batch * seq_q] token rows of n_heads_q heads, k and v are [batch *
 * seq_k] token rows of n_heads_k heads (n_heads_q a multiple of n_heads_k:
 * query head h reads key head h / (n_heads_q / n_heads_k)).  Per sample b and
 * head h, over the keys j that query i sees,
 *
 *     s[i,j] = scale * sum_d q[i,d] * k[j,d]
 *     lse[i] = log sum_j exp(s[i,j]),   p[i,j] = exp(s[i,j] - lse[i])
 *     o[i,d] = sum_j p[i,j] * v[j,d]
 *
 * Query i sees key j when j < k_lens[b], i < q_lens[b] (a NULL array: the
 * whole sequence) and, with causal, j <= i + k_lens[b] - q_lens[b] (the
 * diagonal ends at the last valid query and the last valid key).  A query
 * that sees no key answers o = 0 and lse = -inf.  What lies in rows past the
 * lengths, NaN and infinities included, reaches no output.  (Within the
 * lengths a masked key has p = 0, which does not stop a NaN or an infinity: one
 * in a key or value may reach the queries of the same tile that the causal mask
 * hides it from, one in a query or its gradient the gradients of such keys.)
 *
 * The backward pass takes do = dL/do with the forward pass's o and lse and
 * recomputes p:
 *
 *     delta[i] = sum_d do[i,d] * o[i,d]
 *     ds[i,j]  = p[i,j] * (sum_d do[i,d] * v[j,d] - delta[i])
 *     dq[i,d]  = scale * sum_j ds[i,j] * k[j,d]
 *     dk[j,d]  = scale * sum_i ds[i,j] * q[i,d]    (and over the query heads
 *     dv[j,d]  = sum_i p[i,j] * do[i,d]             of a shared key head)
 *
 * A call of at most 16 queries per sample reads every key and value once for
 * all queries of a key head; longer ones take 256-query tiles.
 *
 * Products run on the tensor cores with fp32 accumulators; p and ds enter
 * their second product rounded to the activation dtype, times powers of two
 * that keep them in its range (ds in fp16: taken from |do| and |v|, so that
 * neither small nor large gradients are lost); outputs are rounded once.  No
 * atomics: equal calls give equal bits.
 *
 * Ownership and errors follow qknr.h: the caller owns every buffer (the
 * workspace included), the library allocates nothing and never
 * synchronises; argument errors return before any CUDA call; a bounded
 * in-kernel wait that runs out writes QKNR_ERR_TIMEOUT to *dev_status.
 */
#ifndef QKNR_ATTN_H_
#define QKNR_ATTN_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qknr_attn_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* activations and gradients: QKNR_BF16 or QKNR_FP16 */
  const void *q, *k, *v;      /* device token rows */
  void *o;                    /* forward: written; backward: the forward pass's */
  float *lse;                 /* device [batch, n_heads_q, seq_q]; likewise */
  int64_t q_stride, k_stride, v_stride, o_stride;   /* elements per row; 0 = heads * D */
  int32_t batch, seq_q, seq_k;
  int32_t n_heads_q, n_heads_k, head_dim;           /* head_dim D: 64 or 128 */
  const int32_t *q_lens, *k_lens;                   /* device [batch], or NULL; values are clamped to 0 .. seq */
  float scale;                /* 0 = 1 / sqrt(D) */
  int32_t causal;
  /* backward only */
  const void *dout;           /* do */
  void *dq, *dk, *dv;
  int64_t dout_stride, dq_stride, dk_stride, dv_stride;
  void *workspace;            /* device, 16-byte aligned */
  size_t workspace_bytes;
  int32_t *dev_status;        /* optional device int32 (see qknr.h) */
  uint32_t flags;             /* QKNR_FLAG_NO_OVERLAP, QKNR_FLAG_TEST_STALL */
  uint64_t wait_limit_ns;     /* 0 = 2 s */
} qknr_attn_args;

/* Defaults: bf16, scale 1 / sqrt(D), no mask, everything else zero. */
void qknr_attn_args_init(qknr_attn_args *a);

/* Device bytes the forward (the backward) pass needs at `workspace`; may be
   0.  Pointers are not looked at. */
qknr_status qknr_attn_workspace_bytes(const qknr_attn_args *args, size_t *bytes);
qknr_status qknr_attn_backward_workspace_bytes(const qknr_attn_args *args, size_t *bytes);

/* Validate and launch on `stream` (asynchronous).  Base addresses and row
   strides must be 16-byte aligned (lse and the lengths: 4-byte); an output
   must not share an element with an input or another output (columns of one
   buffer may interleave). */
qknr_status qknr_attn_forward(const qknr_attn_args *args, qknr_stream_t stream);
qknr_status qknr_attn_backward(const qknr_attn_args *args, qknr_stream_t stream);

/* sizeof(qknr_attn_args) as compiled into the library. */
size_t qknr_attn_sizeof_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_ATTN_H_ */
