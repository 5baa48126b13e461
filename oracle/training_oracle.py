"""Plain fp64 CPU oracle of the training operators: layer norm and its
gradients, the gradients of the per-head RMSNorm + RoPE, and attention and its
gradients.

TEST INFRASTRUCTURE.  Only the tests and the smoke check use this module; it
shares no code with the CUDA library.  Inputs are fp64 arrays (the values the
device buffers hold); results are unrounded.  The gradients are the formulas'
and are themselves held against central differences of the forward functions.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# layer norm

def _gain(weight, T, rows_per_batch, unit):
    if weight is None:
        return 1.0
    set_of = np.arange(T) // (rows_per_batch or max(T, 1))
    return unit + np.atleast_2d(weight)[set_of]


def layer_norm(x, weight, bias, eps, rows_per_batch=0, unit=0.0):
    """(y, mean, rstd) of rows x [T, C]."""
    T = x.shape[0]
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * _gain(weight, T, rows_per_batch, unit)
    if bias is not None:
        y = y + _gain(bias, T, rows_per_batch, 0.0)
    return y, mean, rstd


def layer_norm_backward(dy, x, weight, mean, rstd, rows_per_batch=0, unit=0.0):
    """(dx, dweight [B, C], dbias [B, C]) for the given mean and rstd."""
    T, C = x.shape
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * _gain(weight, T, rows_per_batch, unit)
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xhat * (g * xhat).mean(1, keepdims=True))
    rpb = rows_per_batch or max(T, 1)
    sets = -(-T // rpb) if rows_per_batch else 1
    dw, db = np.zeros((sets, C)), np.zeros((sets, C))
    for b in range(sets):
        rows = slice(b * rpb, min(T, (b + 1) * rpb))
        dw[b], db[b] = (dy[rows] * xhat[rows]).sum(0), dy[rows].sum(0)
    return dx, dw, db


# ---------------------------------------------------------------------------
# per-head RMSNorm + RoPE

def rope_pairs(D, style):
    """(first, second): the dimensions of each rotation pair's members."""
    if style == "rotate_half":
        return np.arange(D // 2), np.arange(D // 2, D)
    return np.arange(0, D, 2), np.arange(1, D, 2)


def qk_norm_rope(x, gamma, cos, sin, eps, style):
    """x [T, H, D]; cos and sin [T, D] or [T, H, D]."""
    D = x.shape[-1]
    if cos.ndim == 2:
        cos, sin = cos[:, None], sin[:, None]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    a, b = rope_pairs(D, style)
    o = np.empty_like(y)
    o[..., a] = y[..., a] * cos[..., a] - y[..., b] * sin[..., a]
    o[..., b] = y[..., b] * cos[..., b] + y[..., a] * sin[..., b]
    return o


def qk_norm_rope_backward(do, x, gamma, cos, sin, eps, style):
    """(dx [T, H, D], dgamma [D])."""
    D = x.shape[-1]
    if cos.ndim == 2:
        cos, sin = cos[:, None], sin[:, None]
    a, b = rope_pairs(D, style)
    dy = np.empty_like(do)
    dy[..., a] = do[..., a] * cos[..., a] + do[..., b] * sin[..., b]
    dy[..., b] = do[..., b] * cos[..., b] - do[..., a] * sin[..., a]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dy * gamma
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    return dx, (dy * x * r).sum((0, 1))


# ---------------------------------------------------------------------------
# attention: q [B, Sq, Hq, D], k and v [B, Sk, Hk, D]

def visible(Sq, Sk, q_len, k_len, causal):
    """[Sq, Sk]: query i sees key j.  With causal the diagonal ends at the
    last valid query and the last valid key."""
    i, j = np.arange(Sq)[:, None], np.arange(Sk)[None, :]
    m = (i < q_len) & (j < k_len)
    return m & (j <= i + k_len - q_len) if causal else m


def _each(q, k, q_lens, k_lens, causal):
    B, Sq, Hq, _ = q.shape
    Sk, Hk = k.shape[1], k.shape[2]
    for b in range(B):
        m = visible(Sq, Sk, Sq if q_lens is None else q_lens[b], Sk if k_lens is None else k_lens[b], causal)
        for h in range(Hq):
            yield b, h, h // (Hq // Hk), m


def attention(q, k, v, scale, causal=False, q_lens=None, k_lens=None):
    """(o [B, Sq, Hq, D], lse [B, Hq, Sq]); a row that sees no key answers
    zero, with lse -inf.  Keys that a row does not see are not read."""
    B, Sq, Hq, D = q.shape
    o, lse = np.zeros_like(q), np.full((B, Hq, Sq), -np.inf)
    for b, h, hk, m in _each(q, k, q_lens, k_lens, causal):
        rows = np.flatnonzero(m.any(1))
        cols = np.flatnonzero(m.any(0))
        if rows.size == 0:
            continue
        mm = m[np.ix_(rows, cols)]
        s = np.where(mm, q[b, rows, h] @ k[b, cols, hk].T * scale, -np.inf)
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        lse[b, h, rows] = top[:, 0] + np.log(p.sum(1))
        o[b, rows, h] = p @ v[b, cols, hk] / p.sum(1, keepdims=True)
    return o, lse


def attention_backward(do, q, k, v, o, lse, scale, causal=False, q_lens=None, k_lens=None):
    """(dq, dk, dv) for the given o and lse."""
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, h, hk, m in _each(q, k, q_lens, k_lens, causal):
        rows, cols = np.flatnonzero(m.any(1)), np.flatnonzero(m.any(0))
        if rows.size == 0:
            continue
        mm = m[np.ix_(rows, cols)]
        qq, kk, vv, dd = q[b, rows, h], k[b, cols, hk], v[b, cols, hk], do[b, rows, h]
        p = np.where(mm, np.exp(np.where(mm, qq @ kk.T * scale, 0.0) - lse[b, h, rows][:, None]), 0.0)
        delta = (dd * o[b, rows, h]).sum(1, keepdims=True)
        ds = p * (dd @ vv.T - delta) * scale
        dq[b, rows, h] = ds @ kk
        dk[b, cols, hk] += ds.T @ qq
        dv[b, cols, hk] += p.T @ dd
    return dq, dk, dv
