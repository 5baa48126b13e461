"""Nothing is written behind a workspace of exactly the bytes that the library
asks for, and the results are right on it, over every way the work is shared
out."""
import ctypes

import numpy as np
import pytest
import torch

import tests.test_attention_packed_gpu as P
import tests.test_attention_prefix_gpu as X
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.gpu_util import TORCH

pytestmark = pytest.mark.gpu

GUARD = 4 << 20


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


class Exact:
    """A workspace of the bytes that `query` answers, 0xA5 behind it."""

    def __init__(self, query, args):
        n = ctypes.c_size_t(0)
        assert query(ctypes.byref(args), ctypes.byref(n)) == Q.OK
        self.buf = torch.full((n.value + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.buf[:n.value] = 255
        self.n = n.value

    def __enter__(self):
        return self.buf[:self.n] if self.n else None

    def __exit__(self, *_):
        assert (self.buf[self.n:] == 0xA5).all(), "written behind the workspace"


def packed(s, backward):
    lib, td = Q.load(), TORCH[s["dtype"]]
    args = Q.pack_args(s["q"], s["k"], s["v"], s["Hq"], s["Hk"], s["D"], P.ints(s["sq"]), None if s["one"] else P.ints(s["sk"]),
                       causal=s["causal"])
    o, lse = P.kept(*s["q"].shape, dtype=td), P.kept(s["Hq"], s["q"].shape[0])
    with Exact(lib.qknr_pack_workspace_bytes, args) as ws:
        P.call(s, out=o, lse=lse, workspace=ws)
    P.check_forward(s, o, lse)
    if backward:
        grads = [P.kept(*t.shape, dtype=td) for t in (s["q"], s["k"], s["v"])]
        with Exact(lib.qknr_pack_backward_workspace_bytes, args) as ws:
            P.call_backward(s, s["do"], o, lse, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws)
        P.check_backward(s, o, lse, *grads)


# a few queries over few keys, in more tiles than two a CTA: equal shares that cut some
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k,Hq,Hk", [([1] * 20, [900] + [5] * 19, 16, 16), ([1] * 32, [512] * 2 + [0] * 30, 12, 12),
                                                 ([0] * 30 + [1, 1], [0] * 30 + [900, 100], 20, 20), ([1] * 12, [385] + [50] * 11, 96, 48),
                                                 ([2] * 20, [50] * 19 + [70], 16, 16), ([3, 0, 5] * 10, [900] + [4] * 29, 20, 5)])
def test_short_keys_of_many_heads(lens_q, lens_k, Hq, Hk, causal, D, dtype):
    packed(P.make(lens_q, lens_k, Hq, Hk, D, dtype=dtype, causal=causal, seed=81), backward=False)


@pytest.mark.parametrize("seed", range(24))
def test_packed_at_random(seed):
    gen = np.random.Generator(np.random.PCG64(500 + seed))
    B = int(gen.integers(1, 60 if seed % 2 else 8))
    few = seed % 3 == 0
    lens = gen.integers(0, int(gen.choice([60, 400, 1500])) // (3 if B > 8 else 1) + 1, size=B).tolist()
    Hk, group, D = int(gen.integers(1, 9)), int(gen.choice([1, 2])), int(gen.choice([64, 128]))
    s = P.make([min(n, 3) for n in lens] if few else lens, lens if few else None, Hk * group, Hk, D, causal=bool(seed & 4),
               dtype="fp16" if seed & 8 else "bf16", seed=seed)
    if s["q"].shape[0]:
        packed(s, backward=True)


@pytest.mark.parametrize("seed", range(16))
def test_prefix_at_random(seed):
    gen = np.random.Generator(np.random.PCG64(600 + seed))
    B, Sq = int(gen.choice([1, 3, 20, 50])), int(gen.choice([1, 1, 3, 40, 150]))
    Sk, n = int(gen.choice([0, 40, 300, 1100])), int(gen.choice([0, 100, 1000, 4000]))
    Hk, group, D = int(gen.integers(1, 9)), int(gen.choice([1, 2])), int(gen.choice([64, 128]))
    s = X.make(B, Sq, Sk, n, Hk * group, Hk, D, causal=bool(seed & 4), dtype="fp16" if seed & 8 else "bf16", seed=seed)
    args = Q.prefix_args(s["q"], s["k"], s["v"], s["pk"], s["pv"], s["Hq"], s["Hk"], D, batch=B, causal=s["causal"])
    with Exact(Q.load().qknr_prefix_workspace_bytes, args) as ws:
        o, lse = X.call(s, workspace=ws)
    X.check(s, o, lse)


@pytest.mark.parametrize("T,C,rpb", [(1, 64, 0), (700, 1536, 0), (1000, 9088, 333), (37, 32768, 0), (304, 512, 2), (2000, 2048, 0)])
def test_rms_norm_gradients(T, C, rpb):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dy = (torch.randn(T, C, device="cuda", generator=gen).bfloat16() for _ in range(2))
    w = torch.randn(-(-T // rpb) if rpb else 1, C, device="cuda", generator=gen)
    _, rstd, _ = Q.rms_norm(x, w, rows_per_batch=rpb or None)
    args = Q.rms_args(x, w, rows_per_batch=rpb or None)
    with Exact(Q.load().qknr_rms_workspace_bytes, args) as ws:
        a = Q.rms_norm_backward(dy, x, w, rstd, rows_per_batch=rpb or None, workspace=ws)
    b = Q.rms_norm_backward(dy, x, w, rstd, rows_per_batch=rpb or None)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
