"""Packed sequences are apart: nothing that one holds changes a bit of another's
results, and fp16's gradients keep their precision beside values near the end of
the type's range (bounds: test_attention_gradient_range_gpu)."""
import numpy as np
import pytest
import torch

import tests.test_attention_gradient_range_gpu as G
import tests.test_attention_packed_gpu as P
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.training_util import normal, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


# tiles worked out by the CTAs; by the plan, whole; by the plan, cut
LISTS = [([200, 90, 310], 1), ([40] * 20 + [600] + [7] * 20, 20), ([1500, 3200, 20], 0)]


@pytest.mark.parametrize("lens,bad", LISTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("what", ["large", "inf", "nan"])
def test_another_sequence_changes_no_bit(what, dtype, D, lens, bad):
    s = P.make(lens, None, 4, 2, D, dtype=dtype, causal=True, seed=71)
    o, lse = P.call(s)
    grads = P.call_backward(s, s["do"], o, lse)
    rows = slice(s["sq"][bad], s["sq"][bad + 1])
    keep = P.outside(s["q"].shape[0], [rows])
    do = s["do"].clone()
    if what == "large":
        s["v"][rows] *= 10000
        do[rows] *= 30
    else:
        for t in (s["v"], do) if what == "inf" else (s["q"], s["k"], s["v"], do):
            t[rows] = float(what)
    o2, lse2 = P.call(s)
    assert same_bits(o2[keep], o[keep]) and same_bits(lse2[:, keep], lse[:, keep])
    for a, b in zip(P.call_backward(s, do, o2, lse2), grads):
        assert torch.isfinite(a[keep].float()).all() and same_bits(a[keep], b[keep])


@pytest.mark.parametrize("lens,bad", LISTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("v", [30000.0, float("inf")])
@pytest.mark.parametrize("do", [1e-5, 1e-3])
def test_small_gradients_beside_large_values(do, v, D, lens, bad):
    s = P.make(lens, lens, 2, 1, D, dtype="fp16", size=2.0 ** -10, scale=2.0 ** 20 / np.sqrt(D), seed=72)
    gen = np.random.Generator(np.random.PCG64(73))
    s["do"] = normal(gen, s["do"].shape, torch.float16, do)
    s["v"] = normal(gen, s["v"].shape, torch.float16)
    s["v"][s["sk"][bad]:s["sk"][bad + 1]] = v
    o, lse = P.call(s)
    grads = P.call_backward(s, s["do"], o, lse)
    for i, (one, rows, keys) in enumerate(P.each(s)):
        if i != bad and i < bad + 3:
            G.check(dict(one, do=s["do"][rows]), "fp16", o[rows], lse[:, rows], grads[0][rows], grads[1][keys], grads[2][keys])
