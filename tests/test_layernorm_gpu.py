"""Layer norm and its backward pass against the fp64 oracle.

Bounds.  An fp32 sum of n terms added in a tree of depth k is off by at most
k * 2^-24 * sum |terms| (to first order).  A row's sums have a depth of at
most 8 (a thread's chunk) * 8 (its chunks) + 5 (shuffles) + 32 (warps), and
each term carries a few roundings of its own: 128 covers both.  A sum over
rows adds, per thread, the rows of its share, then groups, then partial sums;
256 covers the tests' sizes.  The result is rounded once more into the
output's type."""
import numpy as np
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import training_oracle as R
from tests.gpu_util import TORCH
from tests.training_util import U, f64, half_step, normal, same_bits, smallest, within

pytestmark = pytest.mark.gpu

ROW, ROWS = 128 * U, 256 * U


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    yield
    assert Q.read_status() == 0


def make(T, C, dtype="bf16", param="fp32", sets=1, seed=0, weight=True, bias=True, scale=2.0, offset=0.3):
    g = np.random.Generator(np.random.PCG64(seed))
    pt = torch.float32 if param == "fp32" else TORCH[dtype]
    shape = (C,) if sets == 1 else (sets, C)
    return dict(x=normal(g, (T, C), TORCH[dtype], scale, offset), dy=normal(g, (T, C), TORCH[dtype], 0.3),
                weight=normal(g, shape, pt, 0.5, 0.7) if weight else None,
                bias=normal(g, shape, pt, 0.5) if bias else None)


def check_forward(s, dtype, y, mean, rstd, rpb=0, unit=False, eps=1e-6):
    x, w = f64(s["x"]), None if s["weight"] is None else f64(s["weight"])
    b = None if s["bias"] is None else f64(s["bias"])
    ref, m, r = R.layer_norm(x, w, b, float(np.float32(eps)), rpb, float(unit))
    size = np.abs(x).mean(1)
    within(mean, m, ROW * size, "mean")
    # var is off by ROW of itself, and by the square of the mean's error
    slack = ROW + 2 * ROW * size * r
    within(rstd, r, r * slack, "rstd")
    plain, _, _ = R.layer_norm(x, w, None, float(np.float32(eps)), rpb, float(unit))
    gain = R._gain(w, x.shape[0], rpb, float(unit))
    bound = half_step(dtype) * np.abs(ref) + smallest(dtype) + slack[:, None] * (np.abs(plain) + np.abs(gain)) + 4 * U * np.abs(ref)
    within(y, ref, bound, "y")


def check_backward(s, dtype, mean, rstd, dx, dw, db, rpb=0, unit=False):
    x, dy, w = f64(s["x"]), f64(s["dy"]), None if s["weight"] is None else f64(s["weight"])
    m, r = f64(mean), f64(rstd)
    ref, rw, rb = R.layer_norm_backward(dy, x, w, m, r, rpb, float(unit))
    g = np.abs(dy * R._gain(w, x.shape[0], rpb, float(unit)))
    # xhat is (x - mean) * rstd: off by 2 U of itself (x - mean rounds once)
    xh = np.abs((x - m[:, None]) * r[:, None])
    size = r[:, None] * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    within(dx, ref, half_step(dtype) * np.abs(ref) + smallest(dtype) + ROW * size, "dx")
    _, aw, ab = R.layer_norm_backward(np.abs(dy), m[:, None] + xh / r[:, None], w, m, r, rpb, float(unit))
    within(dw, rw, ROWS * aw, "dweight")
    within(db, rb, ROWS * ab, "dbias")


def both(T, C, dtype="bf16", param="fp32", rpb=0, unit=False, seed=0, **kw):
    sets = -(-T // rpb) if rpb else 1
    s = make(T, C, dtype, param, sets, seed, **kw)
    opt = dict(rows_per_batch=rpb or None, unit_offset=unit)
    y, mean, rstd = Q.layer_norm(s["x"], s["weight"], s["bias"], **opt)
    check_forward(s, dtype, y, mean, rstd, rpb, unit)
    dx, dw, db = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, **opt)
    check_backward(s, dtype, mean, rstd, dx, dw, db, rpb, unit)
    return s, (y, mean, rstd), (dx, dw, db)


@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("bf16", "act"), ("fp16", "fp32"), ("fp16", "act")])
@pytest.mark.parametrize("C", [8, 64, 248, 256, 264, 520, 1000, 1536, 2056, 5120, 8192, 8200, 12288, 16392, 32768])
def test_hidden_sizes(C, dtype, param):
    both(37, C, dtype, param, seed=C)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 151, 152, 153, 611, 1001, 4099])
@pytest.mark.parametrize("C", [64, 1536])
def test_row_counts(T, C):
    both(T, C, seed=T)


@pytest.mark.parametrize("T,rpb", [(6, 1), (10, 3), (700, 1), (1000, 333), (1000, 7), (304, 2), (500, 499), (5, 9)])
@pytest.mark.parametrize("C", [64, 2048, 9000])
def test_samples(T, rpb, C):
    # parameter rows per sample: one row each, a short last sample, more
    # samples than CTAs, about as many
    both(T, C, "bf16", "act", rpb, True, seed=T + rpb)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("unit", [False, True])
def test_missing_parameters(weight, bias, unit):
    both(70, 384, weight=weight, bias=bias, unit=unit, seed=7)


def test_mean_far_from_zero():
    # rows whose mean is a hundred times their spread
    both(50, 1024, "fp16", seed=8, scale=0.5, offset=50.0)


def test_constant_rows():
    x = torch.full((3, 256), 1.5, dtype=torch.bfloat16, device="cuda")
    b = torch.arange(256, dtype=torch.float32, device="cuda")
    y, mean, rstd = Q.layer_norm(x, None, b)
    assert torch.equal(y, b.to(torch.bfloat16).expand(3, -1))
    assert torch.equal(mean, torch.full_like(mean, 1.5))
    torch.testing.assert_close(rstd, torch.full_like(rstd, 1e3), rtol=1e-6, atol=0)


def test_a_nan_stays_in_its_row():
    s = make(9, 512, seed=9)
    y0, m0, r0 = Q.layer_norm(s["x"], s["weight"], s["bias"])
    s["x"][4, 17] = float("nan")
    y, mean, rstd = Q.layer_norm(s["x"], s["weight"], s["bias"])
    assert torch.isnan(y[4]).all() and torch.isnan(mean[4]) and torch.isnan(rstd[4])
    keep = [i for i in range(9) if i != 4]
    assert same_bits(y[keep], y0[keep]) and same_bits(mean[keep], m0[keep])


def test_strided_rows_and_in_place():
    s = make(130, 640, seed=10)
    wide = torch.full((130, 1024), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:704] = s["x"]
    ref = Q.layer_norm(s["x"], s["weight"], s["bias"])
    out = torch.full_like(wide, 5.0)
    got = Q.layer_norm(wide[:, 64:704], s["weight"], s["bias"], out=out[:, 128:768])
    assert all(same_bits(a, b) for a, b in zip(got, ref))
    assert bool((out[:, :128] == 5).all()) and bool((out[:, 768:] == 5).all())
    x = s["x"].clone()
    assert Q.layer_norm(x, s["weight"], s["bias"], out=x)[0] is x and same_bits(x, ref[0])
    dref = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], ref[1], ref[2])
    dy = torch.full_like(wide, 3.0)
    dy[:, 8:648] = s["dy"]
    view = dy[:, 8:648]
    got = Q.layer_norm_backward(view, wide[:, 64:704], s["weight"], ref[1], ref[2], out=view)
    assert all(same_bits(a, b) for a, b in zip(got, dref))
    assert bool((dy[:, :8] == 3).all()) and bool((dy[:, 648:] == 3).all())


def test_equal_calls_give_equal_bits():
    for T, C, rpb in ((1001, 5120, 0), (900, 768, 100), (64, 9216, 0)):
        s, fwd, bwd = both(T, C, rpb=rpb, seed=11)
        for _ in range(3):
            again = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], fwd[1], fwd[2], rows_per_batch=rpb or None)
            assert all(same_bits(a, b) for a, b in zip(again, bwd))


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd = Q.layer_norm(x, w, w)
    assert y.shape == (0, 64) and mean.numel() == 0
    dw, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    Q.layer_norm_backward(x, x, w, mean, rstd, dweight=dw, dbias=db)
    assert float(dw.abs().sum() + db.abs().sum()) == 0.0


def test_on_another_stream_and_in_a_graph():
    s, fwd, bwd = both(777, 1536, seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = Q.layer_norm(s["x"], s["weight"], s["bias"], stream=side)
    got += Q.layer_norm_backward(s["dy"], s["x"], s["weight"], got[1], got[2], stream=side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(got, fwd + bwd))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = Q.layer_norm(s["x"], s["weight"], s["bias"])
        out = (y, mean, rstd) + Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
    for t in out:
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(same_bits(a, b) for a, b in zip(out, fwd + bwd))
