"""Plain fp64 CPU oracle of the root-mean-square norm with the residual's
addition, its 8-bit form and its gradients.

TEST INFRASTRUCTURE.  Only the tests use this module; it shares no code with
the CUDA library.  Inputs are fp64 arrays (the values the device buffers
hold); results are unrounded.  The gradients are the formulas' and are
themselves held against central differences of the forward function.
"""
from __future__ import annotations

import numpy as np

F8_MAX, SCALE_MIN = 448.0, 2.0 ** -126


def gain(weight, T, rows_per_batch=0, unit=0.0):
    """[T, C] or a number."""
    if weight is None:
        return 1.0
    return unit + np.atleast_2d(weight)[np.arange(T) // (rows_per_batch or max(T, 1))]


def rms_norm(x, residual, weight, eps, rows_per_batch=0, unit=0.0):
    """(y, rstd, h) of rows x [T, C]."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gain(weight, x.shape[0], rows_per_batch, unit), rstd, h


def quantize(y, block=0):
    """(y / scale unrounded, scales [T] or [T, C / block])."""
    T, C = y.shape
    parts = y.reshape(T, -1, block or C)
    scales = np.maximum(np.abs(parts).max(2) / F8_MAX, SCALE_MIN)
    return (parts / scales[..., None]).reshape(T, C), scales if block else scales[:, 0]


def rms_norm_backward(dy, x, weight, rstd, dsum=None, rows_per_batch=0, unit=0.0):
    """(dx, dweight [B, C]) for the given rstd."""
    T, C = x.shape
    xhat = x * rstd[:, None]
    g = dy * gain(weight, T, rows_per_batch, unit)
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    rpb = rows_per_batch or max(T, 1)
    dw = np.stack([(dy * xhat)[t:t + rpb].sum(0) for t in range(0, max(T, 1), rpb)])
    return dx if dsum is None else dx + dsum, dw
