"""Gradients of packed attention whose o and lse run over more keys than the
call has (keys split over calls, own keys beside a prefix): every call gives its
keys' part, a query that sees a single one of them included.  Against the fp64
oracle for the same o and lse, with the bounds of attention itself."""
import numpy as np
import pytest
import torch

import tests.test_attention_packed_gpu as P
from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import sequence_oracle as S
from tests.gpu_util import TORCH
from tests.training_util import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


def joint(first, second):
    """o and lse over the keys of both calls."""
    s, D = first, first["D"]
    rows = s["q"].shape[0]
    H = lambda t, h: f64(t).reshape(-1, h, D)  # noqa: E731
    o, lse = np.zeros((rows, s["Hq"], D)), np.full((s["Hq"], rows), -np.inf)
    parts = [S.sequences(x["sq"], x["sk"], rows, x["k"].shape[0]) for x in (first, second)]
    for ((a, b), (c, d)), (_, (e, f)) in zip(*parts):
        n = b - a
        mask = np.concatenate([S.R.visible(n, d - c, n, d - c, first["causal"]), S.R.visible(n, f - e, n, f - e, second["causal"])], 1)
        k, v = (np.concatenate([H(first[x][c:d], s["Hk"]), H(second[x][e:f], s["Hk"])]) for x in "kv")
        o[a:b], lse[:, a:b] = S.masked(H(s["q"][a:b], s["Hq"]), k, v, s["scale"], mask)
    return (torch.from_numpy(o.reshape(rows, -1)).to(TORCH[s["dtype"]]).cuda(), torch.from_numpy(lse).float().cuda())


def part(s, o, lse):
    grads = [P.kept(*t.shape, dtype=TORCH[s["dtype"]]) for t in (s["q"], s["k"], s["v"])]
    P.call_backward(s, s["do"], o, lse, dq=grads[0], dk=grads[1], dv=grads[2])
    P.check_backward(s, o, lse, *grads)
    return grads


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens_q,lens_a,lens_b,causal", [
    ([70, 1, 200], [1, 1, 1], [300, 5, 129], False),      # one key, and the others
    ([1, 3, 2], [1, 40, 1], [1, 1, 700], False),
    ([130, 300, 1], [90, 1, 33], [130, 300, 1], True),    # a prefix, and own keys whose first query sees one
    ([257, 12], [400, 1], [100, 12], True),               # and queries that see none of their own
])
def test_parts_of_a_gradient(lens_q, lens_a, lens_b, causal, D, dtype):
    first = P.make(lens_q, lens_a, 4, 2, D, dtype=dtype, seed=61)
    second = dict(P.make(lens_q, lens_b, 4, 2, D, dtype=dtype, causal=causal, seed=62), q=first["q"], do=first["do"])
    o, lse = joint(first, second)
    a, b = part(first, o, lse), part(second, o, lse)
    # the queries that see one key of a call get a gradient through it
    for s, grads in ((first, a), (second, b)):
        for (x, y), (c, d) in S.sequences(s["sq"], s["sk"], s["q"].shape[0], s["k"].shape[0]):
            if d - c == 1:
                assert grads[0][x:y].float().any(1).all() and grads[1][c:d].float().any()
            elif s["causal"] and 0 <= (y - x) - (d - c):
                assert grads[0][y - (d - c)].float().any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("small", [0.001, 0.02])
def test_values_elsewhere_far_longer(small, D):
    # fp16: dP - delta is as large as the other call's rows of v, not this one's
    first, second = (P.make([150, 9], lens, 2, 1, D, dtype="fp16", seed=seed) for lens, seed in (([5, 1], 64), ([130, 40], 65)))
    second.update(q=first["q"], do=first["do"])
    first["v"] *= small
    first["k"] *= 0.3
    second["k"] *= 0.3
    second["v"] *= 20
    o, lse = joint(first, second)
    part(first, o, lse)
    part(second, o, lse)


@pytest.mark.parametrize("size", [0.05, 1.0, 6.0])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("lens_q,lens_k", [([200, 1, 140], [1, 1, 1]), ([200, 1, 140], None), ([2, 1, 16], [1, 1, 1])])
def test_a_single_key_of_its_own_still_has_none(lens_q, lens_k, dtype, D, size):
    # scores up to about 400, and sums of large terms that cancel
    s = P.make(lens_q, lens_k, 4, 2, D, dtype=dtype, causal=lens_k is None, size=size, seed=63)
    o, lse = P.call(s)
    dq, dk, _ = P.call_backward(s, s["do"], o, lse)
    if lens_k is None:
        assert not any(dq[a].float().any() for a in s["sq"][:-1])
    else:
        assert not dq.float().any() and not dk.float().any()
