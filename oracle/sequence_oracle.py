"""Plain fp64 CPU oracle of attention over packed sequences and beside a shared
prefix: both are attention of single samples, cut out and masked here.

TEST INFRASTRUCTURE.  Only the tests use this module; it shares no code with
the CUDA library.
"""
from __future__ import annotations

import numpy as np

from oracle import training_oracle as R


def bounds(starts, rows):
    """[(first, end)] of each sequence as the starts are read: clamped to the
    rows there are, and a falling one counts as the largest before it."""
    s = np.maximum.accumulate(np.clip(np.asarray(starts, dtype=np.int64), 0, rows))
    return list(zip(s[:-1], s[1:]))


def sequences(starts_q, starts_k, rows_q, rows_k):
    return list(zip(bounds(starts_q, rows_q), bounds(starts_k, rows_k)))


def packed(q, k, v, scale, causal, starts_q, starts_k):
    """(o, lse [Hq, rows]) of rows q [rows, Hq, D]; NaN where a row belongs to
    no sequence."""
    o, lse = np.full(q.shape, np.nan), np.full((q.shape[1], q.shape[0]), np.nan)
    for (a, b), (c, d) in sequences(starts_q, starts_k, len(q), len(k)):
        o1, l1 = R.attention(q[None, a:b], k[None, c:d], v[None, c:d], scale, causal)
        o[a:b], lse[:, a:b] = o1[0], l1[0]
    return o, lse


def packed_backward(do, q, k, v, o, lse, scale, causal, starts_q, starts_k):
    dq, dk, dv = (np.full(t.shape, np.nan) for t in (q, k, v))
    for (a, b), (c, d) in sequences(starts_q, starts_k, len(q), len(k)):
        g = R.attention_backward(do[None, a:b], q[None, a:b], k[None, c:d], v[None, c:d], o[None, a:b], lse[None, :, a:b], scale,
                                 causal)
        dq[a:b], dk[c:d], dv[c:d] = (t[0] for t in g)
    return dq, dk, dv


def prefix_mask(seq_q, seq_k, prefix, q_len, k_len, causal):
    """[seq_q, prefix + seq_k]: query i sees key j of the prefix and its own."""
    own = R.visible(seq_q, seq_k, q_len, k_len, causal)
    return np.concatenate([np.repeat(np.arange(seq_q)[:, None] < q_len, prefix, 1), own], 1)


def masked(q, k, v, scale, mask):
    """(o [n, Hq, D], lse [Hq, n]) of one sample's rows under a mask [n, m];
    keys that nobody sees are not read."""
    n, Hq, _ = q.shape
    group = Hq // k.shape[1]
    o, lse = np.zeros_like(q), np.full((Hq, n), -np.inf)
    rows, cols = np.flatnonzero(mask.any(1)), np.flatnonzero(mask.any(0))
    if rows.size:
        m = mask[np.ix_(rows, cols)]
        for h in range(Hq):
            s = np.where(m, q[rows, h] @ k[cols, h // group].T * scale, -np.inf)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            lse[h, rows] = top[:, 0] + np.log(p.sum(1))
            o[rows, h] = p @ v[cols, h // group] / p.sum(1, keepdims=True)
    return o, lse
