"""The operators of sequences in the checked build (each plain global access
tested against its buffer's span), and with offsets past 2^31 elements.
Addresses that TMA works out are bounded by the tensor maps; what a store puts
outside its rows shows in the rows around them, which hold a value of their
own."""
import numpy as np
import pytest
import torch

import tests.test_attention_packed_gpu as TP
import tests.test_attention_prefix_gpu as TX
import tests.test_rms_gpu as TR
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.test_training_checked_gpu import checked, libs, wide  # noqa: F401  (fixtures)
from tests.training_util import same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,C,rpb", [(1, 8, 0), (3, 264, 1), (700, 1000, 0), (611, 1536, 100), (1001, 5120, 0), (40, 8320, 7),
                                     (5, 32768, 2), (620, 16384, 0)])
@pytest.mark.parametrize("dtype,param,residual", [("bf16", "fp32", True), ("fp16", "act", False)])
def test_rms_norm_stays_in_bounds(checked, T, C, rpb, dtype, param, residual):  # noqa: F811
    TR.all_forms(T, C, dtype, param, rpb, rpb > 0, residual=residual)


@pytest.mark.parametrize("lens_q,lens_k", [([1], None), ([77, 41, 28, 46], None), ([129, 0, 300, 5], None), ([1500, 3, 700], None),
                                           ([300, 64], [5, 2000]), ([1, 1, 1], [500, 0, 3000]), ([2] * 300, None)])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_attention_stays_in_bounds(checked, lens_q, lens_k, D, dtype, causal):  # noqa: F811
    TP.both(lens_q, lens_k, 4, 2, D, dtype=dtype, causal=causal, before=5, behind=40)


@pytest.mark.parametrize("bad", [[0, 300, 100, 450], [-5, 300, 450, 10 ** 9], [2 ** 31 - 1, 0, 5, 0]])
def test_bad_starts_stay_in_bounds(checked, bad):  # noqa: F811
    TP.test_starts_out_of_order_or_range(bad)


@pytest.mark.parametrize("B,Sq,Sk,P", [(1, 1, 1, 1), (3, 7, 300, 129), (64, 1, 100, 3000), (5, 300, 200, 700), (40, 3, 900, 5000),
                                       (16, 40, 64, 4000)])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_prefix_attention_stays_in_bounds(checked, B, Sq, Sk, P, D, dtype):  # noqa: F811
    k_lens = [(i * 37) % (Sk + 1) for i in range(B)]
    TX.run(B, Sq, Sk, P, 6, 2, D, dtype=dtype, causal=True, k_lens=k_lens, seed=B)


def test_checked_build_gives_the_regular_bits(libs, monkeypatch):  # noqa: F811
    s, n = TP.make([700, 30, 1200], None, 4, 2, 64, causal=True, seed=3), TR.make(700, 1536, seed=4)
    x = TX.make(50, 1, 64, 3000, 8, 2, 128, seed=5)

    def results():
        o, lse = TP.call(s)
        y, rstd, h = Q.rms_norm(n["x"], n["weight"], residual=n["residual"])
        q = Q.rms_norm_quantized(n["x"], n["weight"], residual=n["residual"], block=128)
        return [o, lse, *TP.call_backward(s, s["do"], o, lse), y, rstd, h, *q, *Q.rms_norm_backward(n["dy"], h, n["weight"], rstd),
                *TX.call(x)]

    regular = results()
    monkeypatch.setattr(Q, "_lib", libs[1])
    monkeypatch.setattr(Q, "_plans", {})
    assert all(same_bits(a, b) for a, b in zip(regular, results()))
    assert Q.read_status() == 0


def test_rms_norm_past_2_31_elements(wide):  # noqa: F811
    s = TR.make(1200, 512, seed=21)
    got = Q.rms_norm(s["x"], s["weight"], residual=s["residual"])
    back = Q.rms_norm_backward(s["dy"], got[2], s["weight"], got[1], dsum=s["dsum"])
    far = Q.rms_norm(wide(s["x"]), s["weight"], residual=wide(s["residual"]), out=wide(s["x"] * 0), sum_out=wide(s["x"] * 0))
    far_back = Q.rms_norm_backward(wide(s["dy"]), far[2], s["weight"], far[1], dsum=wide(s["dsum"]), out=wide(s["x"] * 0))
    assert all(same_bits(a, b) for a, b in zip((*got, *back), (*far, *far_back)))


@pytest.mark.parametrize("lens,D,causal", [([700, 20, 480], 128, False), ([300, 0, 600, 300], 64, True)])
def test_packed_attention_past_2_31_elements(wide, lens, D, causal):  # noqa: F811
    s = TP.make(lens, None, 2, 1, D, causal=causal, seed=23)
    o, lse = TP.call(s)
    grads = TP.call_backward(s, s["do"], o, lse)
    far = dict(s, q=wide(s["q"]), k=wide(s["k"]), v=wide(s["v"]))
    o2, lse2 = TP.call(far, out=wide(s["q"] * 0))
    assert same_bits(o, o2) and same_bits(lse, lse2)
    got = TP.call_backward(far, wide(s["do"]), o2, lse2, dq=wide(s["q"] * 0), dk=wide(s["k"] * 0), dv=wide(s["v"] * 0))
    assert all(same_bits(a, b) for a, b in zip(grads, got))


@pytest.mark.parametrize("B,Sq,Sk,P", [(24, 1, 40, 1100), (4, 250, 200, 300)])
def test_prefix_attention_past_2_31_elements(wide, B, Sq, Sk, P):  # noqa: F811
    s = TX.make(B, Sq, Sk, P, 2, 1, 64, seed=24)
    o, lse = TX.call(s)
    far = dict(s, **{n: wide(s[n]) for n in ("q", "k", "v", "pk", "pv")})
    o2, lse2 = TX.call(far, out=wide(s["q"] * 0))
    assert same_bits(o, o2) and same_bits(lse, lse2)


def test_a_long_cache_past_2_31_elements():
    # a single query over a packed cache whose elements pass 2^31: its last sequence lies behind them
    rows, D = 17_000_000, 128
    k, v = (torch.empty(rows, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(i))
            for i in (1, 2))
    q = torch.empty(3, 2 * D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(3))
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    at = [0, 1000, rows - 700, rows]
    o, lse = Q.attention_packed(q, k, v, 2, 1, D, ints([0, 1, 2, 3]), ints(at))
    for b in (0, 2):
        part = slice(at[b], at[b + 1])
        o1, lse1 = Q.attention_packed(q[b:b + 1], k[part].clone(), v[part].clone(), 2, 1, D, ints([0, 1]), ints([0, at[b + 1] - at[b]]))
        assert (o[b:b + 1].float() - o1.float()).abs().max() <= 2.0 ** -8 * np.sqrt(2) and (lse[:, b:b + 1] - lse1).abs().max() < 1e-5
    # and the long one in between: its values' mean is near zero, its log-sum near the log of its length plus half a variance
    assert o[1].float().abs().max() < 1e-2 and abs(float(lse[0, 1]) - np.log(at[2] - at[1])) < 2
