"""The norm's oracle against hand values and against central differences."""
import numpy as np
import pytest
import torch

from oracle import rms_oracle as R


def test_a_row_by_hand():
    y, rstd, h = R.rms_norm(np.array([[1.0, 2.0]]), np.array([[2.0, 2.0]]), np.array([2.0, -1.0]), 0.0)
    assert np.allclose(h, [[3.0, 4.0]]) and np.allclose(rstd, [1 / np.sqrt(12.5)])
    assert np.allclose(y, [[6 / np.sqrt(12.5), -4 / np.sqrt(12.5)]])
    v, s = R.quantize(y)
    assert np.allclose(v[0, 0], 448.0) and np.allclose(v * s[:, None], y)


def test_against_torch():
    g = np.random.Generator(np.random.PCG64(0))
    x, w = g.normal(size=(5, 24)), g.normal(size=24)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (24,), torch.from_numpy(w), 1e-5).numpy()
    assert np.allclose(R.rms_norm(x, None, w, 1e-5)[0], ref, atol=1e-12)


@pytest.mark.parametrize("rpb,unit", [(0, 0.0), (2, 1.0)])
def test_gradients_against_differences(rpb, unit):
    g = np.random.Generator(np.random.PCG64(1))
    T, C, eps, step = 5, 8, 1e-3, 1e-5
    x, r, w = g.normal(size=(T, C)), g.normal(size=(T, C)), g.normal(size=(3, C) if rpb else (C,))
    dy, ds = g.normal(size=(T, C)), g.normal(size=(T, C))

    def loss(x, r, w):
        y, _, h = R.rms_norm(x, r, w, eps, rpb, unit)
        return (y * dy).sum() + (h * ds).sum()

    _, rstd, h = R.rms_norm(x, r, w, eps, rpb, unit)
    dx, dw = R.rms_norm_backward(dy, h, w, rstd, ds, rpb, unit)
    for t, c in ((0, 0), (2, 5), (4, 7)):
        e = np.zeros((T, C))
        e[t, c] = step
        assert abs((loss(x + e, r, w) - loss(x - e, r, w)) / (2 * step) - dx[t, c]) < 1e-7
        assert abs((loss(x, r + e, w) - loss(x, r - e, w)) / (2 * step) - dx[t, c]) < 1e-7
    for i in range(w.size):
        e = np.zeros(w.size)
        e[i] = step
        e = e.reshape(w.shape)
        assert abs((loss(x, r, w + e) - loss(x, r, w - e)) / (2 * step) - dw.reshape(-1)[i]) < 1e-7
