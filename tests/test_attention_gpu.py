"""Attention and its backward pass against the fp64 oracle.

Bounds, from the roundings the kernels make (u = 2^-24, h = half a step of
the activation type, t = half a step among its smallest values):

* A score is a tensor-core product of D terms: off by 2 D u of the sum of the
  terms' sizes (twice the rounded sum's bound, as the products' accumulator
  may truncate), and the exponent's argument rounds twice more.  e_p is the
  relative error of p from that and from ex2.approx (2^-22).
* p (and ds) is rounded to the activation type before its second product:
  h of itself, or t where it is tiny.
* A sum over n keys (queries) adds 2 n u of the terms' sizes.
* The output is rounded once more: h of itself, or t.
"""
import numpy as np
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import training_oracle as R
from tests.gpu_util import TORCH
from tests.training_util import U, f64, half_step, normal, same_bits, smallest, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


def split(t, B, H, D):
    return f64(t).reshape(B, -1, H, D)


def score_error(q, k, scale):
    """Bound on |s| 's error per (b, h, i, j), and e_p's part that does not
    depend on the row's log-sum."""
    aq, ak = np.abs(q).transpose(0, 2, 1, 3), np.abs(k).transpose(0, 2, 3, 1)
    size = scale * (aq @ ak)
    return (2 * q.shape[-1] + 4) * U * size


def spread(x, group):
    return np.repeat(x, group, axis=2)


def check_forward(s, dtype, o, lse):
    B, Hq, Hk, D, scale = s["B"], s["Hq"], s["Hk"], s["D"], s["scale"]
    q, k, v = split(s["q"], B, Hq, D), split(s["k"], B, Hk, D), split(s["v"], B, Hk, D)
    masks = (s["causal"], s["q_lens"], s["k_lens"])
    k, v = clean(k, s["k_lens"]), clean(v, s["k_lens"])
    q = clean(q, s["q_lens"])
    ref, rl = R.attention(q, k, v, scale, *masks)
    av, _ = R.attention(q, k, np.abs(v), scale, *masks)
    n = k.shape[1]
    es = score_error(q, spread(k, Hq // Hk), scale).max(3, initial=0.0)              # [B, Hq, Sq]
    ep = 2 * (es + 2.0 ** -22) + (2 * n + 16) * U
    h = half_step(dtype)
    bound = h * np.abs(ref) + (h + ep.transpose(0, 2, 1)[..., None]) * av + smallest(dtype) * (1 + np.abs(v).sum(1).max())
    within(o, ref.reshape(f64(o).shape), bound.reshape(f64(o).shape), "o")
    got = f64(lse).reshape(rl.shape)
    np.testing.assert_array_equal(np.isinf(got), np.isinf(rl))
    fin = np.isfinite(rl)
    assert np.all(np.abs(got[fin] - rl[fin]) <= (es + 2.0 ** -22 + (n + 16) * U + 4 * U * np.abs(np.where(fin, rl, 0)))[fin])


def clean(x, lens):
    """Values past the lengths do not count."""
    if lens is None:
        return x
    x = x.copy()
    for b, n in enumerate(lens):
        x[b, n:] = 0
    return x


def check_backward(s, dtype, do, o, lse, dq, dk, dv):
    B, Hq, Hk, D, scale = s["B"], s["Hq"], s["Hk"], s["D"], s["scale"]
    g = Hq // Hk
    q, k, v = split(s["q"], B, Hq, D), split(s["k"], B, Hk, D), split(s["v"], B, Hk, D)
    dd, oo, ll = split(do, B, Hq, D), split(o, B, Hq, D), f64(lse).reshape(B, Hq, -1)
    q, dd, oo = clean(q, s["q_lens"]), clean(dd, s["q_lens"]), clean(oo, s["q_lens"])
    k, v = clean(k, s["k_lens"]), clean(v, s["k_lens"])
    masks = (s["causal"], s["q_lens"], s["k_lens"])
    rq, rk, rv = R.attention_backward(dd, q, k, v, oo, ll, scale, *masks)
    Sq, Sk = q.shape[1], k.shape[1]
    h, t = half_step(dtype), smallest(dtype)
    bq, bk, bv = np.zeros_like(rq), np.zeros_like(rk), np.zeros_like(rv)
    es = score_error(q, spread(k, g), scale)
    for b, hh, hk, m in R._each(q, k, s["q_lens"], s["k_lens"], s["causal"]):
        l = np.where(np.isfinite(ll[b, hh]), ll[b, hh], 0)[:, None]
        e = es[b, hh] + 2.0 ** -21 + 8 * U * np.abs(l)
        p = np.where(m, np.exp(np.where(m, q[b, :, hh] @ k[b, :, hk].T * scale, -1e30) - l), 0)
        dp, adp = dd[b, :, hh] @ v[b, :, hk].T, np.abs(dd[b, :, hh]) @ np.abs(v[b, :, hk]).T
        delta = (dd[b, :, hh] * oo[b, :, hh]).sum(1, keepdims=True)
        adelta = np.abs(dd[b, :, hh] * oo[b, :, hh]).sum(1, keepdims=True)
        ds = p * (dp - delta)
        eds = p * (e + 4 * U) * (np.abs(dp) + np.abs(delta)) + p * 2 * D * U * (adp + adelta) + h * np.abs(ds) + t * m
        eds = eds * (1 + h) + 2 * max(Sq * g, Sk) * U * np.abs(ds)
        evp = (p * (e + h + 2 * Sq * g * U) + t * m)
        bq[b, :, hh] += scale * eds @ np.abs(k[b, :, hk])
        bk[b, :, hk] += scale * eds.T @ np.abs(q[b, :, hh])
        bv[b, :, hk] += evp.T @ np.abs(dd[b, :, hh])
    for got, ref, bound, name in ((dq, rq, bq, "dq"), (dk, rk, bk, "dk"), (dv, rv, bv, "dv")):
        bound = (bound + h * np.abs(ref) + t) * (1 + 2 * h)
        within(got, ref.reshape(f64(got).shape), bound.reshape(f64(got).shape), name)


def make(B, Sq, Sk, Hq, Hk, D, dtype="bf16", causal=False, q_lens=None, k_lens=None, scale=None, seed=0, packed=False,
         size=1.0, garbage=True):
    gen = np.random.Generator(np.random.PCG64(seed))
    td = TORCH[dtype]
    if packed:
        buf = normal(gen, (B * Sq, (Hq + 2 * Hk) * D), td, size)
        q, k, v = buf[:, :Hq * D], buf[:, Hq * D:(Hq + Hk) * D], buf[:, (Hq + Hk) * D:]
    else:
        q, k, v = (normal(gen, (B * n, H * D), td, size) for n, H in ((Sq, Hq), (Sk, Hk), (Sk, Hk)))
    do = normal(gen, (B * Sq, Hq * D), td, 0.3)
    if garbage:
        # what lies past the lengths is NaN
        for b in range(B):
            if q_lens is not None:
                q[b * Sq + q_lens[b]:(b + 1) * Sq] = float("nan")
                do[b * Sq + q_lens[b]:(b + 1) * Sq] = float("nan")
            if k_lens is not None:
                k[b * Sk + k_lens[b]:(b + 1) * Sk] = float("nan")
                v[b * Sk + k_lens[b]:(b + 1) * Sk] = float("inf")
    return dict(q=q, k=k, v=v, do=do, B=B, Hq=Hq, Hk=Hk, D=D, causal=causal, q_lens=q_lens, k_lens=k_lens,
                scale=1 / np.sqrt(D) if scale is None else float(np.float32(scale)))


def options(s):
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(batch=s["B"], causal=s["causal"], q_lens=dev(s["q_lens"]), k_lens=dev(s["k_lens"]), scale=s["scale"])


def forward(s, **kw):
    return Q.attention(s["q"], s["k"], s["v"], s["Hq"], s["Hk"], s["D"], **options(s), **kw)


def backward(s, o, lse, **kw):
    return Q.attention_backward(s["do"], s["q"], s["k"], s["v"], o, lse, s["Hq"], s["Hk"], s["D"], **options(s), **kw)


def both(*shape, dtype="bf16", **kw):
    s = make(*shape, dtype=dtype, **kw)
    o, lse = forward(s)
    check_forward(s, dtype, o, lse)
    grads = backward(s, o, lse)
    check_backward(s, dtype, s["do"], o, lse, *grads)
    return s, o, lse, grads


SIZES = [(1, 1), (1, 7), (5, 3), (64, 64), (127, 128), (128, 128), (129, 127), (200, 300), (256, 257), (384, 131),
         (515, 640), (1, 700), (700, 1)]


@pytest.mark.parametrize("Sq,Sk", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward_sizes(Sq, Sk, D, dtype):
    s = make(2, Sq, Sk, 2, 2, D, dtype, seed=Sq * 1000 + Sk)
    o, lse = forward(s)
    check_forward(s, dtype, o, lse)


@pytest.mark.parametrize("Sq,Sk", SIZES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_backward_sizes(Sq, Sk, D, dtype):
    both(1, Sq, Sk, 2, 2, D, dtype=dtype, seed=Sq * 1000 + Sk)


@pytest.mark.parametrize("Sq,Sk", SIZES)
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_causal(Sq, Sk, D, dtype):
    # fewer keys than queries: the first rows see nothing
    both(1, Sq, Sk, 2, 1, D, dtype=dtype, causal=True, seed=Sq + Sk)


@pytest.mark.parametrize("Hq,Hk", [(6, 3), (4, 1), (5, 5), (8, 2)])
@pytest.mark.parametrize("causal", [False, True])
def test_shared_key_heads(Hq, Hk, causal):
    both(2, 150, 270, Hq, Hk, 64, causal=causal, seed=Hq)
    both(1, 300, 300, Hq, Hk, 128, causal=causal, seed=Hk, packed=True)


@pytest.mark.parametrize("q_lens,k_lens", [([300, 1, 0, 129], None), (None, [0, 1, 260, 128]), ([128, 257, 3, 300], [260, 5, 129, 0]),
                                           ([0, 0, 0, 0], [0, 0, 0, 0])])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_lengths_with_nan_behind_them(q_lens, k_lens, causal, D, dtype):
    s, o, lse, (dq, dk, dv) = both(4, 300, 260, 2, 1, D, dtype=dtype, causal=causal, q_lens=q_lens, k_lens=k_lens, seed=D)
    for b in range(4):
        if q_lens is not None:
            rows = slice(b * 300 + q_lens[b], (b + 1) * 300)
            assert not o[rows].any() and not dq[rows].any()
            assert bool((lse[b, :, q_lens[b]:] == -float("inf")).all())
        if k_lens is not None:
            rows = slice(b * 260 + k_lens[b], (b + 1) * 260)
            assert not dk[rows].any() and not dv[rows].any()


def test_lengths_outside_the_sequence_are_clamped():
    s = make(2, 70, 90, 1, 1, 64, seed=3)
    ref = forward(s)
    s["q_lens"], s["k_lens"] = [70, 0], [90, 0]
    want = forward(s)
    s["q_lens"], s["k_lens"] = [1 << 30, -5], [91, -(1 << 31)]
    got = forward(s)
    assert all(same_bits(a, b) for a, b in zip(want, got))
    assert same_bits(got[0][:70], ref[0][:70])


@pytest.mark.parametrize("size", [0.01, 4.0, 12.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_flat_and_peaked_rows(size, dtype):
    # logits from nearly equal to hundreds apart (the running maximum moves)
    both(1, 260, 520, 2, 2, 64, dtype=dtype, seed=5, size=size)
    both(1, 130, 390, 1, 1, 128, dtype=dtype, seed=6, size=size, scale=0.2)


def test_rising_scores():
    # every block's largest score is far above the block's before it
    s = make(1, 128, 640, 1, 1, 64, seed=7)
    ramp = torch.arange(640, device="cuda")[:, None] / 640 * 6
    s["k"] = (s["k"] * 0.05 + ramp).to(torch.bfloat16)
    s["q"] = (s["q"] * 0.05 + 1.5).to(torch.bfloat16)
    o, lse = forward(s)
    check_forward(s, "bf16", o, lse)
    check_backward(s, "bf16", s["do"], o, lse, *backward(s, o, lse))


def test_a_nan_stays_in_its_rows():
    s = make(1, 300, 200, 2, 2, 64, seed=8)
    o, lse = forward(s)
    s["q"][40, :64] = float("nan")
    o2, lse2 = forward(s)
    assert torch.isnan(o2[40, :64]).all() and bool(torch.isnan(lse2[0, 0, 40]))
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[40, :64] = False
    assert torch.equal(o[keep], o2[keep])


def test_wide_strides_and_given_outputs():
    s, o, lse, grads = both(2, 190, 190, 3, 1, 64, packed=True, seed=9)
    buf = torch.full((380, 5 * 64 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    dst = [buf[:, 8:200], buf[:, 200:264], buf[:, 264:328]]
    got = backward(s, o, lse, dq=dst[0], dk=dst[1], dv=dst[2])
    assert all(a is b for a, b in zip(got, dst)) and all(same_bits(a, b) for a, b in zip(got, grads))
    assert bool((buf[:, :8] == 7).all()) and bool((buf[:, 328:] == 7).all())
    wide = torch.full((380, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    l2 = torch.empty_like(lse)
    got, _ = forward(s, out=wide[:, 40:232], lse=l2)
    assert same_bits(got, o) and same_bits(l2, lse)
    assert bool((wide[:, :40] == 7).all()) and bool((wide[:, 232:] == 7).all())


def test_equal_calls_give_equal_bits():
    for shape, kw in (((2, 700, 700, 4, 2, 128), dict(causal=True)), ((1, 1, 4100, 6, 3, 64), {})):
        s, o, lse, grads = both(*shape, seed=10, **kw)
        for _ in range(3):
            assert all(same_bits(a, b) for a, b in zip(forward(s), (o, lse)))
            assert all(same_bits(a, b) for a, b in zip(backward(s, o, lse), grads))


def test_many_calls_one_after_the_other():
    # nothing waits between the calls: roles of a CTA drift apart as far as
    # the kernels let them, and every call gives the first one's bits
    for shape, kw in (((2, 300, 260, 3, 1, 64), dict(q_lens=[300, 129], k_lens=[129, 260], causal=True)),
                      ((1, 640, 515, 2, 2, 128), dict(k_lens=[389]))):
        s = make(*shape, dtype="fp16", seed=14, **kw)
        first = forward(s)
        first += backward(s, *first)
        kept = []
        for i in range(300):
            f = forward(s)
            f += backward(s, *f)
            if i % 25 == 0:
                kept.append(f)
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for f in kept for a, b in zip(f, first))


def test_on_another_stream_and_in_a_graph():
    s, o, lse, grads = both(1, 333, 333, 2, 1, 64, causal=True, seed=11, k_lens=[300], q_lens=[310])
    opt = options(s)
    args = (s["q"], s["k"], s["v"])
    heads = (s["Hq"], s["Hk"], s["D"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = Q.attention(*args, *heads, stream=side, **opt)
    got += Q.attention_backward(s["do"], *args, *got, *heads, stream=side, **opt)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, (o, lse) + grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = Q.attention(*args, *heads, **opt)
        out = f + Q.attention_backward(s["do"], *args, *f, *heads, **opt)
    for t in out:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for a, b in zip(out, (o, lse) + grads))


@pytest.mark.parametrize("Sq,Sk", [(0, 5), (5, 0), (0, 0)])
def test_no_queries_or_no_keys(Sq, Sk):
    s = make(2, Sq, Sk, 2, 1, 64, seed=12)
    o, lse = forward(s)
    assert not o.any() and bool((lse == -float("inf")).all())
    dq, dk, dv = backward(s, o, lse)
    assert dq.shape == (2 * Sq, 128) and not dq.any() and not dk.any() and not dv.any()


def test_a_wait_that_runs_out_is_reported():
    s = make(1, 300, 300, 2, 2, 64, seed=13)
    o, lse = forward(s)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=Q.FLAG_TEST_STALL, wait_limit_ns=2_000_000, dev_status=status)
    forward(s, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == Q.ERR_TIMEOUT
    status.zero_()
    backward(s, o, lse, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == Q.ERR_TIMEOUT
    # the context is whole: the next calls are right
    got = forward(s)
    assert same_bits(got[0], o)
