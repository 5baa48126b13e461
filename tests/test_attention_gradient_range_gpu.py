"""Attention's backward pass over the whole range of gradients, fp16 above
all: dS = P (dP - delta) is as small as the gradient over the number of keys
and as large as |do| |v|, far outside what 16 bits of a half hold.

Bounds as in test_attention_gpu, but for dS's rounding near zero.  There the
kernels round 2^kS dS, with 2^14 P (dP - delta) 2^-e < 2^15 for 2^e <= b <
2^(e+1), b = 2 |do| V: half a subnormal step is 2^-25 2^-kS <= 2^-39 b, with b
the query's own for dq and the largest of the sample's key head for dk.  V is
the kernels' bound on the rows of v, the root of each 8 columns' largest sum of
squares, added up.  bf16 has fp32's exponents: 2^-134."""
import numpy as np
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import training_oracle as R
from tests.gpu_util import TORCH
from tests.test_attention_gpu import backward, clean, forward, make, score_error, split, spread
from tests.training_util import U, f64, half_step, normal, same_bits, smallest, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0


def check(s, dtype, o, lse, dq, dk, dv):
    B, Hq, Hk, D, scale = s["B"], s["Hq"], s["Hk"], s["D"], s["scale"]
    g = Hq // Hk
    q, k, v = split(s["q"], B, Hq, D), split(s["k"], B, Hk, D), split(s["v"], B, Hk, D)
    dd, oo, ll = split(s["do"], B, Hq, D), split(o, B, Hq, D), f64(lse).reshape(B, Hq, -1)
    q, dd, oo = clean(q, s["q_lens"]), clean(dd, s["q_lens"]), clean(oo, s["q_lens"])
    k, v = clean(k, s["k_lens"]), clean(v, s["k_lens"])
    refs = R.attention_backward(dd, q, k, v, oo, ll, scale, s["causal"], s["q_lens"], s["k_lens"])
    Sq, Sk = q.shape[1], k.shape[1]
    h, t = half_step(dtype), smallest(dtype)
    bounds = [np.zeros_like(x) for x in refs]
    es = score_error(q, spread(k, g), scale)
    longest = np.sqrt((v ** 2).reshape(-1, D // 8, 8).sum(-1).max(0).sum())
    row = 2 * np.sqrt((dd ** 2).sum(-1)) * longest                                  # [B, Sq, Hq]
    if dtype == "fp16":
        near_q, near_k = 2.0 ** -39 * row, 2.0 ** -39 * row.max(1, keepdims=True).reshape(B, 1, Hk, g).max(-1)
    else:
        near_q, near_k = np.full_like(row, t), np.full((B, 1, Hk), t)
    for b, hh, hk, m in R._each(q, k, s["q_lens"], s["k_lens"], s["causal"]):
        l = np.where(np.isfinite(ll[b, hh]), ll[b, hh], 0)[:, None]
        e = es[b, hh] + 2.0 ** -21 + 8 * U * np.abs(l)
        p = np.where(m, np.exp(np.where(m, q[b, :, hh] @ k[b, :, hk].T * scale, -1e30) - l), 0)
        dp, adp = dd[b, :, hh] @ v[b, :, hk].T, np.abs(dd[b, :, hh]) @ np.abs(v[b, :, hk]).T
        delta = (dd[b, :, hh] * oo[b, :, hh]).sum(1, keepdims=True)
        adelta = np.abs(dd[b, :, hh] * oo[b, :, hh]).sum(1, keepdims=True)
        ds = p * (dp - delta)
        eds = p * (e + 4 * U) * (np.abs(dp) + np.abs(delta)) + p * 2 * D * U * (adp + adelta) + h * np.abs(ds)
        eds = eds * (1 + h) + 2 * max(Sq * g, Sk) * U * np.abs(ds)
        bounds[0][b, :, hh] += scale * (eds + near_q[b, :, hh, None] * m) @ np.abs(k[b, :, hk])
        bounds[1][b, :, hk] += scale * (eds + near_k[b, 0, hk] * m).T @ np.abs(q[b, :, hh])
        bounds[2][b, :, hk] += (p * (e + h + 2 * Sq * g * U) + t * m).T @ np.abs(dd[b, :, hh])
    for got, ref, bound, name in zip((dq, dk, dv), refs, bounds, ("dq", "dk", "dv")):
        bound = (bound + h * np.abs(ref) + t) * (1 + 2 * h)
        within(got, ref.reshape(f64(got).shape), bound.reshape(f64(got).shape), name)


def case(B, Sq, Sk, Hq, Hk, D, dtype, do, v=1.0, logits=-10, seed=0, **kw):
    """q and k of size 2^logits under a scale that keeps the scores near one:
    small ones make dq and dk large, large ones small, whatever dS is."""
    s = make(B, Sq, Sk, Hq, Hk, D, dtype, seed=seed, size=2.0 ** logits, scale=2.0 ** (-2 * logits) / np.sqrt(D), **kw)
    gen = np.random.Generator(np.random.PCG64(seed + 1))
    s["do"] = normal(gen, (B * Sq, Hq * D), TORCH[dtype], do)
    s["v"] = normal(gen, (B * Sk, Hk * D), TORCH[dtype], v)
    return s


def run(s, dtype):
    o, lse = forward(s)
    grads = backward(s, o, lse)
    check(s, dtype, o, lse, *grads)
    return o, lse, grads


@pytest.mark.parametrize("do", [1e-3, 1e-4, 1e-5, 1e-6])
@pytest.mark.parametrize("Sq,Sk,Hq,Hk,D", [(130, 4096, 1, 1, 128), (257, 4000, 2, 1, 64)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_small_gradients_over_many_keys(Sq, Sk, Hq, Hk, D, dtype, do):
    run(case(1, Sq, Sk, Hq, Hk, D, dtype, do, seed=D), dtype)


@pytest.mark.parametrize("do,v", [(3000.0, 100.0), (3000.0, 1.0), (1.0, 10000.0), (1e-4, 3000.0)])
@pytest.mark.parametrize("causal", [False, True])
def test_large_products(do, v, causal):
    # |do| |v| up to 3e8: far above 65504, with gradients that are not
    run(case(1, 300, 300, 2, 1, 128, "fp16", do, v, logits=6, seed=7, causal=causal), "fp16")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Sq,Sk,Hq,Hk,D", [(700, 900, 4, 2, 64), (1024, 1024, 2, 2, 128)])
def test_rows_heads_and_samples_of_unlike_size(Sq, Sk, Hq, Hk, D, causal):
    # samples and heads a thousand times apart; every other query a hundred
    # thousand times smaller than its neighbours, some with no gradient
    s = case(2, Sq, Sk, Hq, Hk, D, "fp16", 1.0, seed=9, causal=causal)
    do = s["do"].view(2, Sq, Hq, D)
    do[1] *= 1e-3
    do[:, :, :Hq // 2] *= 1e-3
    do[:, ::2] *= 1e-5
    do[:, 5::7] = 0
    run(s, "fp16")


def test_lengths_with_nan_behind_them():
    # neither the queries' nor the values' rows past the lengths count for the factor
    s = case(3, 300, 400, 2, 2, 64, "fp16", 1e-4, seed=11, q_lens=[300, 129, 0], k_lens=[260, 400, 7])
    for b in range(3):
        s["do"][b * 300 + s["q_lens"][b]:(b + 1) * 300] = float("nan")
        s["v"][b * 400 + s["k_lens"][b]:(b + 1) * 400] = float("inf")
        s["v"][b * 400 + s["k_lens"][b]:(b + 1) * 400:2] = 60000.0
    run(s, "fp16")


@pytest.mark.parametrize("what", ["do", "v", "both"])
def test_nothing_to_scale(what):
    s = case(1, 200, 300, 2, 1, 64, "fp16", 1.0, seed=12)
    for name in ("do", "v") if what == "both" else (what,):
        s[name].zero_()
    o, lse, (dq, dk, dv) = run(s, "fp16")
    assert not dq.any() and not dk.any()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk,D", [(1, 300, 700, 2, 1, 64), (2, 515, 515, 2, 2, 128), (1, 5, 2000, 4, 1, 64),
                                             (1, 4096, 4096, 2, 2, 64)])
def test_powers_of_two_pass_through(B, Sq, Sk, Hq, Hk, D, causal):
    # do times 2^-12, exact: every product and sum is the same but for its
    # exponent, so the gradients are too where a half can say so
    s = case(B, Sq, Sk, Hq, Hk, D, "fp16", 1.0, seed=13, causal=causal)
    s["do"] = (s["do"] * 8).round().clamp(-15, 15) / 8
    o, lse = forward(s)
    big = backward(s, o, lse)
    s["do"] = s["do"] * 2.0 ** -12
    small = backward(s, o, lse)
    for a, b in zip(big, small):
        want = a.double() * 2.0 ** -12
        assert bool(((b.double() - want).abs() <= 2.0 ** -25).all())
        exact = want.abs() >= 2.0 ** -14          # normal halves
        assert torch.equal(b.double()[exact], want[exact])
    assert bool((big[0].abs() >= 2.0 ** -2).any())
    again = backward(s, o, lse)
    assert all(same_bits(a, b) for a, b in zip(small, again))
