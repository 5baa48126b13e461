"""The training operators in the checked build (each plain global access
tested against its buffer's span), past 2^31 elements, and with waits that run
out.  Addresses that TMA works out are bounded by the tensor maps; what a
store puts outside its rows shows in the padding around them."""
import numpy as np
import pytest
import torch

import tests.test_attention_gpu as TA
import tests.test_layernorm_gpu as TL
import tests.test_qk_grad_gpu as TG
from diffusion_transformer_qk_gb300 import build as B
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.training_util import same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def libs(built_lib, cuda_device):
    return Q.load(), Q.load(B.ensure_built(checked=True))


@pytest.fixture
def checked(libs, monkeypatch):
    monkeypatch.setattr(Q, "_lib", libs[1])
    monkeypatch.setattr(Q, "_plans", {})
    Q.status_buffer().zero_()
    yield
    torch.cuda.synchronize()
    assert Q.read_status() == 0, "the checked build found an access outside a buffer"


@pytest.mark.parametrize("T,C,rpb", [(1, 8, 0), (3, 264, 1), (700, 1000, 0), (611, 1536, 100), (1001, 5120, 0),
                                     (40, 8200, 7), (5, 32768, 2), (620, 16392, 0)])
@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("fp16", "act")])
def test_layer_norm_stays_in_bounds(checked, T, C, rpb, dtype, param):
    TL.both(T, C, dtype, param, rpb, rpb > 0)


@pytest.mark.parametrize("T,hq,hk,hv", [(1, 1, 0, 0), (3, 24, 8, 8), (500, 7, 3, 2), (129, 0, 5, 1), (1000, 3, 3, 0)])
@pytest.mark.parametrize("D,style", [(64, "rotate_half"), (128, "interleaved")])
@pytest.mark.parametrize("cos_rows", [None, 1])
def test_qk_backward_stays_in_bounds(checked, T, hq, hk, hv, D, style, cos_rows):
    TG.run(T, hq, hk, hv, D, style, cos_rows=cos_rows)
    TG.run(T, hq, hk, hv, D, style, cos_rows=cos_rows, out=False, table="bf16")


@pytest.mark.parametrize("B_,Sq,Sk,Hq,Hk", [(1, 1, 1, 1, 1), (2, 129, 300, 4, 2), (3, 257, 127, 3, 3), (1, 130, 2000, 2, 1),
                                            (1, 3, 1500, 1, 1)])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_stays_in_bounds(checked, B_, Sq, Sk, Hq, Hk, D, dtype, causal):
    TA.both(B_, Sq, Sk, Hq, Hk, D, dtype=dtype, causal=causal)


def test_attention_with_lengths_stays_in_bounds(checked):
    TA.both(4, 300, 260, 2, 2, 64, q_lens=[128, 257, 3, 300], k_lens=[260, 5, 129, 0])


def test_checked_build_gives_the_regular_bits(libs, monkeypatch):
    s, l = TA.make(2, 300, 700, 4, 2, 128, seed=3), TL.make(700, 1536, seed=4)

    def results():
        o, lse = TA.forward(s)
        y, mean, rstd = Q.layer_norm(l["x"], l["weight"], l["bias"])
        return [o, lse, *TA.backward(s, o, lse), y, mean, rstd, *Q.layer_norm_backward(l["dy"], l["x"], l["weight"], mean, rstd)]

    regular = results()
    monkeypatch.setattr(Q, "_lib", libs[1])
    monkeypatch.setattr(Q, "_plans", {})
    assert all(same_bits(a, b) for a, b in zip(regular, results()))
    assert Q.read_status() == 0


# ---------------------------------------------------------------------------
# offsets past 2^31 elements: narrow columns of a buffer with very long rows

WIDE = 1 << 21


@pytest.fixture
def wide(cuda_device):
    """Copies of token rows as columns of rows 4 MB apart; the elements next
    to them stay as they were."""
    buf = torch.full((1200, WIDE), 7.0, dtype=torch.bfloat16, device="cuda")       # 5 GB, 2.5e9 elements
    used = [64]

    def place(t):
        n, w = t.shape
        view = buf[:n, used[0]:used[0] + w]
        view.copy_(t)
        used[0] += w + 64
        return view

    yield place
    left = buf[:, :used[0]] == 7.0
    assert left[:, :64].all() and left[:, used[0] - 64:].all()


def test_layer_norm_past_2_31_elements(wide):
    s = TL.make(1200, 512, seed=21)
    y, mean, rstd = Q.layer_norm(s["x"], s["weight"], s["bias"])
    dx, dw, db = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
    x, dy, out, gx = wide(s["x"]), wide(s["dy"]), wide(s["x"] * 0), wide(s["x"] * 0)
    y2, m2, r2 = Q.layer_norm(x, s["weight"], s["bias"], out=out)
    got = Q.layer_norm_backward(dy, x, s["weight"], m2, r2, out=gx)
    for a, b in zip((y, mean, rstd, dx, dw, db), (y2, m2, r2, *got)):
        assert same_bits(a, b)


def test_qk_backward_past_2_31_elements(wide):
    (dx, dgq, dgk), (dout, qkv, gq, gk, cos, sin, kw) = TG.run(1200, 2, 2, 1, 64, "interleaved", seed=22)
    got = Q.qk_norm_rope_packed_backward(wide(dout), wide(qkv), 2, 2, 1, 64, gq, gk, cos, sin, out=wide(dout * 0), **kw)
    for a, b in zip((dx, dgq, dgk), got):
        assert same_bits(a, b)


@pytest.mark.parametrize("B_,S,D,causal", [(1, 1200, 128, False), (4, 300, 64, True)])
def test_attention_past_2_31_elements(wide, B_, S, D, causal):
    s = TA.make(B_, S, S, 2, 1, D, causal=causal, seed=23)
    o, lse = TA.forward(s)
    grads = TA.backward(s, o, lse)
    far = dict(s, q=wide(s["q"]), k=wide(s["k"]), v=wide(s["v"]), do=wide(s["do"]))
    o2, lse2 = TA.forward(far, out=wide(s["q"] * 0))
    assert same_bits(o, o2) and same_bits(lse, lse2)
    got = TA.backward(far, o2, lse2, dq=wide(s["q"] * 0), dk=wide(s["k"] * 0), dv=wide(s["v"] * 0))
    for a, b in zip(grads, got):
        assert same_bits(a, b)


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,C", [(1000, 1536), (700, 8200)])
def test_layer_norm_waits_that_run_out_are_reported(T, C):
    s = TL.make(T, C, seed=31)
    y, mean, rstd = Q.layer_norm(s["x"], s["weight"], s["bias"])
    dx, dw, db = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=Q.FLAG_TEST_STALL, wait_limit_ns=2_000_000, dev_status=status)
    Q.layer_norm(s["x"], s["weight"], s["bias"], **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == Q.ERR_TIMEOUT
    status.zero_()
    Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == Q.ERR_TIMEOUT
    # the context is whole: the next calls are right
    again = Q.layer_norm(s["x"], s["weight"], s["bias"]) + Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd)
    for a, b in zip((y, mean, rstd, dx, dw, db), again):
        assert same_bits(a, b)
