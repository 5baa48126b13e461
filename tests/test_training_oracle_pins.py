"""The fp64 oracle of the training operators against what its formulas fix:
gradients equal central differences of the forward functions, and the masks'
and layouts' edge cases hold."""
import numpy as np
import pytest

from oracle import qknr_oracle as O
from oracle import training_oracle as R

H = 1e-6      # step of the differences: error ~ H^2 + 1e-16 / H per unit, 1e-9 relative


def differences(f, x):
    """Central differences of the scalar f at each element of x."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + H
        a = f()
        x[i] = old - H
        b = f()
        x[i] = old
        g[i] = (a - b) / (2 * H)
    return g


def close(a, b):
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("rows_per_batch,unit", [(0, 0.0), (2, 1.0), (3, 0.0)])
def test_layer_norm_gradients_are_differences(rows_per_batch, unit):
    g = np.random.Generator(np.random.PCG64(1))
    T, C = 5, 8
    sets = -(-T // rows_per_batch) if rows_per_batch else 1
    x, dy = g.normal(size=(T, C)), g.normal(size=(T, C))
    w, b = g.normal(size=(sets, C)), g.normal(size=(sets, C))

    def loss():
        return (R.layer_norm(x, w, b, 1e-3, rows_per_batch, unit)[0] * dy).sum()

    _, mean, rstd = R.layer_norm(x, w, b, 1e-3, rows_per_batch, unit)
    dx, dw, db = R.layer_norm_backward(dy, x, w, mean, rstd, rows_per_batch, unit)
    close(dx, differences(loss, x))
    close(dw, differences(loss, w))
    close(db, differences(loss, b))


@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
@pytest.mark.parametrize("expanded", [False, True])
def test_qk_gradients_are_differences(style, expanded):
    g = np.random.Generator(np.random.PCG64(2))
    T, heads, D = 3, 2, 8
    x, do, gamma = g.normal(size=(T, heads, D)), g.normal(size=(T, heads, D)), g.normal(size=D)
    shape = (T, heads, D) if expanded else (T, D)
    cos, sin = g.normal(size=shape), g.normal(size=shape)

    def loss():
        return (R.qk_norm_rope(x, gamma, cos, sin, 1e-3, style) * do).sum()

    dx, dgamma = R.qk_norm_rope_backward(do, x, gamma, cos, sin, 1e-3, style)
    close(dx, differences(loss, x))
    close(dgamma, differences(loss, gamma))


@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
def test_qk_forward_is_the_forward_oracles(style):
    g = np.random.Generator(np.random.PCG64(3))
    T, heads, D = 6, 3, 64
    bits = g.integers(0x3f00, 0x4000, size=(T, heads * D)).astype(np.uint16)
    gamma, ang = g.normal(size=D).astype(np.float32), g.normal(size=(T, D))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    ref = O.forward_packed(bits, "bf16", heads, 0, 0, D, gamma, gamma, 1e-6, cos, sin, "fp32", style)["q"]
    got = R.qk_norm_rope(O.decode(bits, "bf16").reshape(T, heads, D), gamma.astype(np.float64),
                         cos.astype(np.float64), sin.astype(np.float64), float(np.float32(1e-6)), style)
    np.testing.assert_allclose(got.reshape(ref.shape), ref, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("causal,q_lens,k_lens", [(False, None, None), (True, None, None), (False, None, [5, 0]),
                                                  (True, [4, 2], [3, 5])])
def test_attention_gradients_are_differences(causal, q_lens, k_lens):
    g = np.random.Generator(np.random.PCG64(4))
    B, Sq, Sk, Hq, Hk, D = 2, 4, 5, 2, 1, 3
    q, do = g.normal(size=(B, Sq, Hq, D)), g.normal(size=(B, Sq, Hq, D))
    k, v = g.normal(size=(B, Sk, Hk, D)), g.normal(size=(B, Sk, Hk, D))

    def loss():
        return (R.attention(q, k, v, 0.7, causal, q_lens, k_lens)[0] * do).sum()

    o, lse = R.attention(q, k, v, 0.7, causal, q_lens, k_lens)
    for got, x in zip(R.attention_backward(do, q, k, v, o, lse, 0.7, causal, q_lens, k_lens), (q, k, v)):
        close(got, differences(loss, x))


def test_rows_that_see_nothing():
    g = np.random.Generator(np.random.PCG64(5))
    q, k, v = g.normal(size=(1, 4, 1, 2)), g.normal(size=(1, 2, 1, 2)), g.normal(size=(1, 2, 1, 2))
    o, lse = R.attention(q, k, v, 1.0, causal=True)
    # four queries, two keys: the last query sees both, the first two none
    assert np.all(o[0, :2] == 0) and np.all(lse[0, 0, :2] == -np.inf) and np.all(np.isfinite(lse[0, 0, 2:]))
    np.testing.assert_array_equal(o[0, 2], v[0, 0])
    # values that no row sees are not read
    k[0, 1], v[0, 1] = np.nan, np.inf
    o2, _ = R.attention(q, k, v, 1.0, k_lens=[1])
    np.testing.assert_array_equal(o2[0], np.broadcast_to(v[0, :1], o2[0].shape))
