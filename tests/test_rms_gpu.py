"""The root-mean-square norm, its 8-bit form and its backward pass against the
fp64 oracle.

Bounds.  x + residual in fp32 is off by U = 2^-24 of itself.  An fp32 sum of n
squares added in a tree of depth k is off by at most k U of itself (a row's
sum: 8 values of a chunk, 8 chunks, 5 shuffles, 32 slots; 128 U covers them
with each term's own roundings), and rsqrt halves that.  A sum over rows adds,
per thread, the rows of its share, then groups, then partial sums; 256 U of
the terms' absolute sum covers the tests' sizes.  A result is rounded once
more into its type: e4m3 by at most 2^-4 of itself, or 2^-10 below 2^-6."""
import numpy as np
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import rms_oracle as R
from tests.gpu_util import TORCH
from tests.training_util import U, f64, half_step, normal, same_bits, smallest, within

pytestmark = pytest.mark.gpu

ROW, ROWS = 128 * U, 256 * U
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    yield
    assert Q.read_status() == 0


def make(T, C, dtype="bf16", param="fp32", sets=0, seed=0, weight=True, residual=True, scale=2.0):
    g = np.random.Generator(np.random.PCG64(seed))
    pt = torch.float32 if param == "fp32" else TORCH[dtype]
    return dict(x=normal(g, (T, C), TORCH[dtype], scale, 0.3), residual=normal(g, (T, C), TORCH[dtype], 1.0) if residual else None,
                weight=normal(g, (sets, C) if sets else (C,), pt, 0.5, 0.7) if weight else None,
                dy=normal(g, (T, C), TORCH[dtype], 0.3), dsum=normal(g, (T, C), TORCH[dtype], 0.3) if residual else None)


def d64(t):
    return None if t is None else f64(t)


def check_forward(s, dtype, y, rstd, h, rpb=0, unit=False):
    ry, rr, rh = R.rms_norm(f64(s["x"]), d64(s["residual"]), d64(s["weight"]), EPS, rpb, float(unit))
    within(rstd, rr, ROW * rr, "rstd")
    if s["residual"] is None:
        assert h is s["x"]
    else:
        within(h, rh, (half_step(dtype) + U) * np.abs(rh) + smallest(dtype), "h")
    within(y, ry, (half_step(dtype) + ROW) * np.abs(ry) + smallest(dtype), "y")
    return ry


def check_quantized(s, y, scales, rstd, h, block, dtype, rpb=0, unit=False):
    ry, rr, rh = R.rms_norm(f64(s["x"]), d64(s["residual"]), d64(s["weight"]), EPS, rpb, float(unit))
    rv, rs = R.quantize(ry, block)
    assert y.dtype == torch.float8_e4m3fn and y.shape == s["x"].shape and scales.shape == rs.shape
    within(rstd, rr, ROW * rr, "rstd")
    within(scales, rs, 2 * ROW * rs, "scales")
    within(y.float(), rv, (2.0 ** -4 + 4 * ROW) * np.abs(rv) + 2.0 ** -10, "y")
    if s["residual"] is not None:
        within(h, rh, (half_step(dtype) + U) * np.abs(rh) + smallest(dtype), "h")


def check_backward(s, dtype, x, rstd, dx, dw, rpb=0, unit=False):
    xx, dy, r, w = f64(x), f64(s["dy"]), f64(rstd), d64(s["weight"])
    ref, rw = R.rms_norm_backward(dy, xx, w, r, d64(s["dsum"]), rpb, float(unit))
    g = np.abs(dy * R.gain(w, xx.shape[0], rpb, float(unit)))
    xh = np.abs(xx * r[:, None])
    size = r[:, None] * (g + xh * (g * xh).mean(1, keepdims=True)) + (0 if s["dsum"] is None else np.abs(f64(s["dsum"])))
    within(dx, ref, half_step(dtype) * np.abs(ref) + smallest(dtype) + ROW * size, "dx")
    if w is None:
        assert dw is None
    else:
        _, aw = R.rms_norm_backward(np.abs(dy), np.abs(xx), w, r, None, rpb, float(unit))
        assert dw.shape == s["weight"].shape
        within(dw, rw, ROWS * aw, "dweight")


def all_forms(T, C, dtype="bf16", param="fp32", rpb=0, unit=False, seed=0, **kw):
    s = make(T, C, dtype, param, -(-T // rpb) if rpb else 0, seed, **kw)
    opt = dict(rows_per_batch=rpb or None, unit_offset=unit)
    y, rstd, h = Q.rms_norm(s["x"], s["weight"], residual=s["residual"], **opt)
    check_forward(s, dtype, y, rstd, h, rpb, unit)
    for block in (None, 128) if C % 128 == 0 else (None,):
        got = Q.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"], block=block, **opt)
        check_quantized(s, *got, block or 0, dtype, rpb, unit)
        assert same_bits(got[2], rstd) and same_bits(got[3], h)
    dx, dw = Q.rms_norm_backward(s["dy"], h, s["weight"], rstd, dsum=s["dsum"], **opt)
    check_backward(s, dtype, h, rstd, dx, dw, rpb, unit)
    return s, (y, rstd, h), (dx, dw)


@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("bf16", "act"), ("fp16", "fp32"), ("fp16", "act")])
@pytest.mark.parametrize("C", [8, 64, 128, 248, 256, 264, 520, 1000, 1536, 2056, 5120, 8192, 8200, 12288, 12416, 16392, 32768])
def test_hidden_sizes(C, dtype, param):
    all_forms(37, C, dtype, param, seed=C)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 151, 152, 153, 607, 608, 609, 1001, 4099])
@pytest.mark.parametrize("C", [64, 384, 1536])
@pytest.mark.parametrize("residual", [True, False])
def test_row_counts(T, C, residual):
    all_forms(T, C, seed=T, residual=residual)


@pytest.mark.parametrize("C", [136, 2048, 6144, 8192, 12288])
@pytest.mark.parametrize("residual", [True, False])
def test_streamed_rows(C, residual):
    all_forms(1301, C, "fp16", "act", seed=C, residual=residual)


@pytest.mark.parametrize("T,rpb", [(6, 1), (10, 3), (700, 1), (1000, 333), (1000, 7), (304, 2), (500, 499), (5, 9)])
@pytest.mark.parametrize("C", [64, 2048, 9088])
def test_samples(T, rpb, C):
    all_forms(T, C, "bf16", "act", rpb, True, seed=T + rpb)


@pytest.mark.parametrize("unit", [False, True])
@pytest.mark.parametrize("residual", [True, False])
def test_no_weight(unit, residual):
    all_forms(70, 384, weight=False, unit=unit, seed=7, residual=residual)


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    y, rstd, h = Q.rms_norm(x, w, residual=x)
    y8, scales, _, _ = Q.rms_norm_quantized(x, w, block=128)
    assert y.shape == h.shape == y8.shape == x.shape and rstd.shape == (0,) and scales.shape == (0, 2)
    dx, dw = Q.rms_norm_backward(x, x, w, rstd)
    assert dx.shape == x.shape and torch.equal(dw, torch.zeros(256, device="cuda"))


def test_zero_rows_and_the_largest_values():
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    x[1] = 65504.0
    x[2, 3] = 65504.0
    x[3] = 6e-8
    s = dict(x=x, residual=None, weight=None, dy=None, dsum=None)
    check_forward(s, "fp16", *Q.rms_norm(x))
    for block in (None, 128):
        got = Q.rms_norm_quantized(x, block=block)
        check_quantized(s, *got, block or 0, "fp16")
        assert torch.equal(got[1][0], torch.full_like(got[1][0], 2.0 ** -126)) and not got[0][0].float().any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_nan_stays_in_its_row(value):
    s = make(700, 512, seed=3)
    clean = Q.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"])
    y0 = Q.rms_norm(s["x"], s["weight"], residual=s["residual"])[0]
    dirty = s["x"].clone()
    dirty[5, 100] = value
    y, scales, rstd, h = Q.rms_norm_quantized(dirty, s["weight"], residual=s["residual"])
    keep = torch.arange(700, device="cuda") != 5
    for a, b in zip((y, scales, rstd), clean):
        assert same_bits(a[keep], b[keep])
    assert y[5].float().isnan().all() and scales[5].isnan()
    if value != value:
        assert rstd[5].isnan()
    assert same_bits(Q.rms_norm(dirty, s["weight"], residual=s["residual"])[0][keep], y0[keep])
    # a scale per block: only the NaN's own block where the statistic is fine (an infinity's rstd is 0)
    yb, sb, _, _ = Q.rms_norm_quantized(dirty, s["weight"], residual=s["residual"], block=128)
    assert sb[5, 0].isnan() and yb[5, :128].float().isnan().all()
    assert sb[5, 1:].isnan().all() == (value != value)


def test_strides_and_in_place():
    g = np.random.Generator(np.random.PCG64(11))
    wide = normal(g, (650, 3 * 512), torch.bfloat16)
    x, r, rest = wide[:, :512], wide[:, 512:1024], wide[:, 1024:].clone()
    w = normal(g, (512,), torch.float32, 0.2, 1.0)
    y0, rstd0, h0 = Q.rms_norm(x.clone(), w, residual=r.clone())
    dy, ds = normal(g, (650, 512), torch.bfloat16), normal(g, (650, 512), torch.bfloat16)
    dx0, dw0 = Q.rms_norm_backward(dy, h0, w, rstd0, dsum=ds)
    y, rstd, h = Q.rms_norm(x, w, residual=r, out=x, sum_out=r)
    assert y is x and h is r
    assert same_bits(y, y0) and same_bits(rstd, rstd0) and same_bits(h, h0) and same_bits(wide[:, 1024:], rest)
    for place in (dy.clone(), ds.clone()):
        first = same_bits(place, dy)
        dx, dw = Q.rms_norm_backward(place if first else dy, r, w, rstd, dsum=ds if first else place, out=place)
        assert dx is place and same_bits(dx, dx0) and same_bits(dw, dw0)
    # 8 bits into the columns of a wider buffer
    f8 = torch.zeros(650, 1024, dtype=torch.float8_e4m3fn, device="cuda")
    a = Q.rms_norm_quantized(h0, w, out=f8[:, 512:])
    b = Q.rms_norm_quantized(h0, w)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and not f8[:, :512].float().any()


def test_equal_calls_give_equal_bits():
    s, fwd, bwd = all_forms(1500, 2048, seed=5)
    for _ in range(3):
        again = Q.rms_norm(s["x"], s["weight"], residual=s["residual"])
        assert all(same_bits(a, b) for a, b in zip(again, fwd))
        assert all(same_bits(a, b) for a, b in zip(Q.rms_norm_backward(s["dy"], fwd[2], s["weight"], fwd[1], dsum=s["dsum"]), bwd))


def test_graph_and_streams():
    s, fwd, bwd = all_forms(900, 1536, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = Q.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"], stream=side)
    side.synchronize()
    with torch.cuda.stream(side):
        assert all(same_bits(a, b) for a, b in zip(q, Q.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"])))
    torch.cuda.synchronize()
    x, dy = s["x"].clone(), s["dy"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, rstd, h = Q.rms_norm(x, s["weight"], residual=s["residual"])
        dx, dw = Q.rms_norm_backward(dy, h, s["weight"], rstd, dsum=s["dsum"])
    for seed in (1, 2):
        g = np.random.Generator(np.random.PCG64(seed))
        x.copy_(normal(g, x.shape, x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        e = Q.rms_norm(x, s["weight"], residual=s["residual"])
        f = Q.rms_norm_backward(dy, e[2], s["weight"], e[1], dsum=s["dsum"])
        assert all(same_bits(a, b) for a, b in zip((y, rstd, h, dx, dw), (*e, *f)))


def test_waits_are_bounded():
    s = make(3000, 512, seed=2)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    rstd = torch.ones(3000, device="cuda")
    kw = dict(flags=Q.FLAG_TEST_STALL, wait_limit_ns=20_000_000, dev_status=word)
    for call in (lambda: Q.rms_norm(s["x"], s["weight"], residual=s["residual"], **kw),
                 lambda: Q.rms_norm_quantized(s["x"], s["weight"], **kw),
                 lambda: Q.rms_norm_backward(s["dy"], s["x"], s["weight"], rstd, dsum=s["dsum"], **kw)):
        word.zero_()
        call()
        assert int(word.item()) == Q.ERR_TIMEOUT
    all_forms(3000, 512, seed=2)


def test_more_than_2_31_elements():
    T, C = 270_000, 8192
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.ones(C, device="cuda")
    y, rstd, _ = Q.rms_norm(x, w)
    y8, scales, _, _ = Q.rms_norm_quantized(x, w, block=128)
    dx, dw = Q.rms_norm_backward(x, x, w, rstd)
    for at in (0, T // 2, T - 3):
        rows = slice(at, at + 3)
        s = dict(x=x[rows], residual=None, weight=w, dy=x[rows], dsum=None)
        check_forward(s, "bf16", y[rows], rstd[rows], s["x"])
        check_quantized(s, y8[rows], scales[rows], rstd[rows], None, 128, "bf16")
        part, _ = Q.rms_norm_backward(x[rows], x[rows], w, rstd[rows])
        assert same_bits(part, dx[rows])
