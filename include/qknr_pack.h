/*
 * qknr_pack.h — C ABI of attention over packed sequences, and its backward
 * pass, in libqknr.so: the operation of qknr_attn.h for a batch whose
 * sequences follow each other without padding.
 *
 * q (and o, do, dq) is [rows_q] token rows of n_heads_q heads, k and v (and
 * dk, dv) [rows_k] token rows of n_heads_k heads.  Sequence b < batch is the
 * query rows q_starts[b] .. q_starts[b + 1] - 1 and the key rows k_starts[b]
 * .. k_starts[b + 1] - 1; the starts are device arrays of batch + 1 values.
 * Formulas, scale, rounding and what a query that sees no key answers are
 * qknr_attn.h's, with q_len = q_starts[b + 1] - q_starts[b] and k_len likewise:
 * with causal, query i of a sequence sees its keys j <= i + k_len - q_len.
 *
 * The backward pass's o and lse may run over more keys than the call has (keys
 * split over calls, own keys beside a prefix): dq, dk and dv are then what its
 * keys add to the gradients.  A query that sees one key and whose lse is that
 * key's score gets exact zeros in dq, as a sequence's only key does in dk: the
 * probability is 1 whatever the score.
 *
 * Starts are clamped to 0 .. rows, and one below an earlier one counts as the
 * largest of them, so that no row belongs to two sequences whatever they say.
 * Rows that belong to no sequence (before the first, behind the last) are
 * neither read into a result nor written: o, lse, dq, dk and dv keep what
 * they held there.
 *
 * Work is shared out on the device by the sequences' lengths.  A call whose
 * sequences have 16 queries or fewer on average takes a sequence's group * q_len
 * query rows of a key head (group = n_heads_q / n_heads_k) 16 at a time, 8 where
 * they are 8 or fewer on average, and reads the sequence's keys and values once
 * for each 16 or 8; other calls take tiles of 256 queries of a head.  The form
 * is the whole call's: long sequences beside many single tokens are better off
 * in a call of their own.
 *
 * No atomics: equal calls give equal bits.  What one sequence's rows hold
 * changes no bit of another's results.
 *
 * Ownership and errors follow qknr.h: the caller owns every buffer (the
 * workspace included), the library allocates nothing and never
 * synchronises; argument errors return before any CUDA call; a bounded
 * in-kernel wait that runs out writes QKNR_ERR_TIMEOUT to *dev_status.
 */
#ifndef QKNR_PACK_H_
#define QKNR_PACK_H_

#include "qknr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct qknr_pack_args {
  uint32_t abi_version;       /* QKNR_ABI_VERSION */
  int32_t dtype;              /* activations and gradients: QKNR_BF16 or QKNR_FP16 */
  const void *q, *k, *v;      /* device token rows */
  void *o;                    /* forward: written; backward: the forward pass's, or a joint one */
  float *lse;                 /* device [n_heads_q, rows_q]; likewise */
  int64_t q_stride, k_stride, v_stride, o_stride;   /* elements per row; 0 = heads * D */
  int32_t batch;              /* sequences; 0: nothing is done */
  int32_t rows_q, rows_k;
  int32_t n_heads_q, n_heads_k, head_dim;           /* head_dim D: 64 or 128 */
  const int32_t *q_starts;    /* device [batch + 1] */
  const int32_t *k_starts;    /* device [batch + 1]; NULL: q_starts */
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
} qknr_pack_args;

/* Defaults: bf16, scale 1 / sqrt(D), no mask, everything else zero. */
void qknr_pack_args_init(qknr_pack_args *a);

/* Device bytes the forward (the backward) pass needs at `workspace`.
   Pointers are not looked at. */
qknr_status qknr_pack_workspace_bytes(const qknr_pack_args *args, size_t *bytes);
qknr_status qknr_pack_backward_workspace_bytes(const qknr_pack_args *args, size_t *bytes);

/* Validate and launch on `stream` (asynchronous).  Alignment and overlap as
   for qknr_attn_forward (the starts: 4-byte aligned). */
qknr_status qknr_pack_forward(const qknr_pack_args *args, qknr_stream_t stream);
qknr_status qknr_pack_backward(const qknr_pack_args *args, qknr_stream_t stream);

/* sizeof(qknr_pack_args) as compiled into the library. */
size_t qknr_pack_sizeof_args(void);

#ifdef __cplusplus
}
#endif

#endif /* QKNR_PACK_H_ */
