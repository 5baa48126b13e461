/*
 * qknr_prefix.h — C ABI of attention for a batch that shares a prefix of keys
 * and values (one prompt, or one reference image, sampled several times), in
 * libqknr.so: the operation of qknr_attn.h where every sample's keys begin
 * with the same `prefix` rows, held once.
 *
 * q and o are [batch * seq_q] token rows of n_heads_q heads, k and v [batch *
 * seq_k] of n_heads_k heads, prefix_k and prefix_v [prefix] of n_heads_k
 * heads.  Query i < q_lens[b] of sample b sees all `prefix` keys, and of its
 * own keys what it sees in qknr_attn.h: j < k_lens[b] and, with causal,
 * j <= i + k_lens[b] - q_lens[b].  lse and o run over both.  A query past
 * q_lens[b] answers o = 0 and lse = -inf, as does one that sees no key.
 *
 * Where the samples' queries are few, those of the whole batch go through the
 * prefix together, and the results of prefix and own keys are joined in fp32;
 * otherwise a tile of queries runs over the prefix and its own keys in one
 * go.  p enters its product rounded to the activation dtype and o is rounded
 * once, as in qknr_attn.h.  No atomics: equal calls give equal bits.
 *
 * Ownership and errors follow qknr.h: the caller owns every buffer (the
 * workspace included), the library allocates nothing and never
 * synchronises; argument errors return before any CUDA call; a bounded
 * in-kernel wait that runs out writes QKNR_ERR_TIMEOUT to *dev_status.
 */
#ifndef QKNR_PREFIX_H_
#define QKNR_PREFIX_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qknr_prefix_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* QKNR_BF16 or QKNR_FP16 */
  const void *q, *k, *v;      /* device token rows */
  const void *prefix_k, *prefix_v;
  void *o;
  float *lse;                 /* device [batch, n_heads_q, seq_q] */
  int64_t q_stride, k_stride, v_stride, prefix_k_stride, prefix_v_stride, o_stride;   /* elements per row; 0 = heads * D */
  int32_t batch, seq_q, seq_k, prefix;              /* seq_k and prefix may be 0 */
  int32_t n_heads_q, n_heads_k, head_dim;           /* head_dim D: 64 or 128 */
  const int32_t *q_lens, *k_lens;                   /* device [batch], or NULL; values are clamped to 0 .. seq */
  float scale;                /* 0 = 1 / sqrt(D) */
  int32_t causal;
  void *workspace;            /* device, 16-byte aligned */
  size_t workspace_bytes;
  int32_t *dev_status;        /* optional device int32 (see qknr.h) */
  uint32_t flags;             /* QKNR_FLAG_NO_OVERLAP, QKNR_FLAG_TEST_STALL */
  uint64_t wait_limit_ns;     /* 0 = 2 s */
} qknr_prefix_args;

/* Defaults: bf16, scale 1 / sqrt(D), no mask, everything else zero. */
void qknr_prefix_args_init(qknr_prefix_args *a);

/* Device bytes needed at `workspace`; may be 0.  Pointers are not looked at. */
qknr_status qknr_prefix_workspace_bytes(const qknr_prefix_args *args, size_t *bytes);

/* Validate and launch on `stream` (asynchronous).  Alignment and overlap as
   for qknr_attn_forward. */
qknr_status qknr_prefix_forward(const qknr_prefix_args *args, qknr_stream_t stream);

/* sizeof(qknr_prefix_args) as compiled into the library. */
size_t qknr_prefix_sizeof_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_PREFIX_H_ */
