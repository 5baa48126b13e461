"""Backward pass of the fused QK-RMSNorm + RoPE against the fp64 oracle.

Bounds.  The two sums over a head are trees of depth 8 + 4, their terms carry
up to 4 roundings, dx combines them with about 8 more: 32 * 2^-24 of the
largest terms' sizes, plus one rounding into the output's type.  dgamma is a
sum over tokens and heads: each lane adds its items in order (at most 200 in
these tests), a CTA's teams add theirs (32), then the partial rows (64)."""
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
    yield
    assert Q.read_status() == 0


def tables(gen, rows, heads, D, table, expanded):
    # any values do (a rotation's or not): the formula takes them as they are
    shape = (rows, heads, D) if expanded else (rows, D)
    dt = torch.float32 if table == "fp32" else torch.bfloat16
    ang = gen.normal(size=shape) * 3
    return torch.from_numpy(np.cos(ang)).to(dt).cuda(), torch.from_numpy(np.sin(ang)).to(dt).cuda()


def check_side(x, do, gamma, cos, sin, style, dtype, H, D, dx, dgamma, eps=1e-6):
    T = x.shape[0]
    rows = np.arange(T) % cos.shape[0]
    c, s = f64(cos)[rows], f64(sin)[rows]
    xx, dd, g = f64(x).reshape(T, H, D), f64(do).reshape(T, H, D), f64(gamma)
    e = float(np.float32(eps))
    ref, rg = R.qk_norm_rope_backward(dd, xx, g, c, s, e, style)
    ac, as_ = (np.abs(c)[:, None], np.abs(s)[:, None]) if c.ndim == 2 else (np.abs(c), np.abs(s))
    a, b = R.rope_pairs(D, style)
    dy = np.empty_like(dd)
    dy[..., a] = np.abs(dd[..., a]) * ac[..., a] + np.abs(dd[..., b]) * as_[..., b]
    dy[..., b] = np.abs(dd[..., b]) * ac[..., b] + np.abs(dd[..., a]) * as_[..., a]
    r = 1 / np.sqrt((xx * xx).mean(-1, keepdims=True) + e)
    gg = dy * np.abs(g)
    size = r * (gg + np.abs(xx) * r * r * (gg * np.abs(xx)).mean(-1, keepdims=True))
    within(dx, ref.reshape(T, H * D), (half_step(dtype) * np.abs(ref) + smallest(dtype) + 32 * U * size).reshape(T, H * D), "dx")
    within(dgamma, rg, 300 * U * (dy * np.abs(xx) * r).sum((0, 1)), "dgamma")


def run(T, hq, hk, hv, D, style, dtype="bf16", table="fp32", expanded=False, cos_rows=None, out=True, seed=0):
    g = np.random.Generator(np.random.PCG64(seed))
    td = TORCH[dtype]
    width = (hq + hk + hv) * D
    qkv, dout = normal(g, (T, width), td, 2.0), normal(g, (T, width), td, 0.3)
    gq, gk = normal(g, (D,), torch.float32, 0.3, 1.0), normal(g, (D,), torch.float32, 0.3, 1.0)
    cos, sin = tables(g, cos_rows or T, hq or hk, D, table, expanded)
    kw = dict(rope_style=style, cos_layout="per_head_expanded" if expanded else "shared_row")
    keep = dout.clone()
    o = torch.full_like(dout, 9.0) if out else None
    dx, dgq, dgk = Q.qk_norm_rope_packed_backward(dout, qkv, hq, hk, hv, D, gq, gk, cos, sin, out=o, **kw)
    q0, k0 = hq * D, (hq + hk) * D
    if hq:
        check_side(qkv[:, :q0], keep[:, :q0], gq, cos, sin, style, dtype, hq, D, dx[:, :q0], dgq)
    if hk:
        check_side(qkv[:, q0:k0], keep[:, q0:k0], gk, cos, sin, style, dtype, hk, D, dx[:, q0:k0], dgk)
    assert same_bits(dx[:, k0:], keep[:, k0:])
    assert (dgq is None) == (hq == 0) and (dgk is None) == (hk == 0)
    if out:
        assert same_bits(dout, keep)
    return (dx, dgq, dgk), (keep, qkv, gq, gk, cos, sin, kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
@pytest.mark.parametrize("dtype,table", [("bf16", "fp32"), ("bf16", "bf16"), ("fp16", "fp32"), ("fp16", "bf16")])
@pytest.mark.parametrize("expanded", [False, True])
def test_forms(D, style, dtype, table, expanded):
    run(61, 5, 5, 3, D, style, dtype, table, expanded, seed=D)


@pytest.mark.parametrize("T,hq,hk,hv", [(1, 1, 0, 0), (1, 0, 1, 1), (3, 24, 8, 8), (2, 1, 1, 0), (500, 7, 3, 2),
                                        (4099, 2, 1, 1), (130, 40, 40, 40)])
@pytest.mark.parametrize("style", ["interleaved", "rotate_half"])
def test_sizes(T, hq, hk, hv, style):
    run(T, hq, hk, hv, 128, style, seed=T)
    run(T, hq, hk, hv, 64, style, "fp16", seed=T, out=False)


@pytest.mark.parametrize("cos_rows", [1, 7, 100, 250])
def test_table_shared_by_samples(cos_rows):
    run(500, 3, 2, 1, 64, "rotate_half", cos_rows=cos_rows, seed=cos_rows)
    run(500, 2, 2, 1, 128, "interleaved", cos_rows=cos_rows, expanded=True, seed=cos_rows)


def test_separate_tensor_equals_packed():
    (dx, dgq, _), (dout, qkv, gq, _, cos, sin, kw) = run(333, 6, 6, 6, 128, "rotate_half", seed=3)
    got, dg = Q.qk_norm_rope_tensor_backward(dout[:, :768], qkv[:, :768], 6, 128, gq, cos, sin,
                                             out=torch.empty_like(dout[:, :768]), **kw)
    assert same_bits(got, dx[:, :768])
    # the same items, summed over the same launch shape
    assert same_bits(dg, dgq)


def test_zero_rows_of_x():
    # r = 1 / sqrt(eps): finite, as in the forward pass
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    d = torch.full((2, 128), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    one, zero = torch.ones((2, 64), device="cuda"), torch.zeros((2, 64), device="cuda")
    dx, dg = Q.qk_norm_rope_tensor_backward(d, x, 2, 64, torch.ones(64, device="cuda"), one, zero, out=torch.empty_like(d))
    assert torch.equal(dx.float(), torch.full_like(dx.float(), 0.9765625)) and float(dg.abs().max()) == 0.0


def test_equal_calls_give_equal_bits_and_a_graph_too():
    (dx, dgq, dgk), (dout, qkv, gq, gk, cos, sin, kw) = run(2048, 8, 4, 4, 64, "interleaved", seed=4)
    out = torch.empty_like(dout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = Q.qk_norm_rope_packed_backward(dout, qkv, 8, 4, 4, 64, gq, gk, cos, sin, out=out, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(got, (dx, dgq, dgk)))


def test_no_rows():
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    t = torch.empty((0, 64), device="cuda")
    _, dg = Q.qk_norm_rope_tensor_backward(x, x, 2, 64, torch.ones(64, device="cuda"), t, t)
    assert float(dg.abs().sum()) == 0.0
