"""Attention beside a shared prefix against the fp64 oracle, with the bounds of
attention itself (tests/test_attention_gpu.py) over prefix and own keys."""
import numpy as np
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import sequence_oracle as S
from tests.gpu_util import TORCH
from tests.training_util import U, f64, half_step, normal, same_bits, smallest, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


def make(B, Sq, Sk, P, Hq, Hk, D, dtype="bf16", causal=False, q_lens=None, k_lens=None, seed=0, size=1.0):
    gen, td = np.random.Generator(np.random.PCG64(seed)), TORCH[dtype]
    q = normal(gen, (B * Sq, Hq * D), td, size)
    kv, shared = normal(gen, (B * Sk, 2 * Hk * D), td, size), normal(gen, (P, 2 * Hk * D), td, size)
    for b in range(B):                # what lies past the lengths
        if q_lens is not None:
            q[b * Sq + q_lens[b]:(b + 1) * Sq] = float("nan")
        if k_lens is not None:
            kv[b * Sk + k_lens[b]:(b + 1) * Sk] = float("nan")
    c = Hk * D
    return dict(q=q, k=kv[:, :c], v=kv[:, c:], pk=shared[:, :c], pv=shared[:, c:], B=B, Sq=Sq, Sk=Sk, P=P, Hq=Hq, Hk=Hk, D=D,
                dtype=dtype, causal=causal, q_lens=q_lens, k_lens=k_lens)


def call(s, **kw):
    dev = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return Q.attention_prefix(s["q"], s["k"], s["v"], s["pk"], s["pv"], s["Hq"], s["Hk"], s["D"], batch=s["B"], causal=s["causal"],
                              q_lens=dev(s["q_lens"]), k_lens=dev(s["k_lens"]), **kw)


def check(s, o, lse):
    B, Sq, Sk, P, Hq, Hk, D = (s[x] for x in ("B", "Sq", "Sk", "P", "Hq", "Hk", "D"))
    scale, h = 1 / np.sqrt(D), half_step(s["dtype"])
    o, lse = f64(o).reshape(B, Sq, Hq, D), f64(lse).reshape(B, Hq, Sq)
    pk, pv = f64(s["pk"]).reshape(P, Hk, D), f64(s["pv"]).reshape(P, Hk, D)
    for b in range(B):
        ql, kl = Sq if s["q_lens"] is None else s["q_lens"][b], Sk if s["k_lens"] is None else s["k_lens"][b]
        mask = S.prefix_mask(Sq, kl, P, ql, kl, s["causal"])
        q = np.nan_to_num(f64(s["q"][b * Sq:(b + 1) * Sq]).reshape(Sq, Hq, D))
        own = slice(b * Sk, b * Sk + kl)
        k = np.concatenate([pk, f64(s["k"][own]).reshape(kl, Hk, D)])
        v = np.concatenate([pv, f64(s["v"][own]).reshape(kl, Hk, D)])
        ref, rl = S.masked(q, k, v, scale, mask)
        av, _ = S.masked(q, k, np.abs(v), scale, mask)
        n = P + kl
        ak = np.abs(np.repeat(k, Hq // Hk, 1)).transpose(1, 2, 0)
        es = ((2 * D + 4) * U * scale * (np.abs(q).transpose(1, 0, 2) @ ak)).max(2, initial=0.0)    # [Hq, Sq]
        ep = 2 * (es + 2.0 ** -22) + (2 * n + 16) * U
        bound = h * np.abs(ref) + (h + ep.T[..., None]) * av + smallest(s["dtype"]) * (1 + np.abs(v).sum(0).max(initial=0.0))
        within(torch.from_numpy(o[b]), ref, bound, f"o of sample {b}")
        np.testing.assert_array_equal(np.isinf(lse[b]), np.isinf(rl))
        fin = np.isfinite(rl)
        assert np.all(np.abs(lse[b][fin] - rl[fin]) <= (es + 2.0 ** -22 + (n + 16) * U + 4 * U * np.abs(np.where(fin, rl, 0)))[fin])


def run(*args, **kw):
    s = make(*args, **kw)
    o, lse = call(s)
    check(s, o, lse)
    return s, o, lse


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp16", 64), ("fp16", 128)])
@pytest.mark.parametrize("P", [1, 127, 128, 129, 1000])
@pytest.mark.parametrize("B,Sq,Sk", [(1, 1, 1), (5, 1, 130), (3, 7, 300), (2, 40, 40), (2, 300, 129), (40, 1, 17), (9, 129, 200)])
def test_sizes(B, Sq, Sk, P, dtype, D):
    run(B, Sq, Sk, P, 4, 2, D, dtype=dtype, seed=P + Sq)


@pytest.mark.parametrize("B,Sq,Sk,P", [(33, 1, 64, 5000), (64, 1, 100, 2000), (20, 2, 30, 9000), (64, 3, 3, 4000), (30, 17, 40, 3000),
                                       (12, 128, 128, 2600), (16, 130, 130, 1500)])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (12, 3), (16, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_long_prefixes(B, Sq, Sk, P, Hq, Hk, causal):
    run(B, Sq, Sk, P, Hq, Hk, 64 if Hq == 12 else 128, causal=causal, seed=P)


@pytest.mark.parametrize("B,Sq,Sk,P", [(6, 1, 90, 700), (6, 20, 90, 700), (6, 300, 400, 700), (6, 5, 90, 20000)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_lengths(B, Sq, Sk, P, causal, dtype):
    # own keys of every length, none among them, and fewer keys than queries
    k_lens, q_lens = [0, 1, Sk, Sk // 2, Sk // 3, 7], [Sq, Sq, Sq // 2, 0, Sq, 1]
    run(B, Sq, Sk, P, 4, 2, 64, dtype=dtype, causal=causal, k_lens=k_lens, seed=1)
    run(B, Sq, Sk, P, 4, 2, 128, dtype=dtype, causal=causal, k_lens=k_lens, q_lens=q_lens, seed=2)


@pytest.mark.parametrize("B,Sq,Sk,P", [(3, 1, 0, 500), (3, 200, 0, 500), (3, 1, 300, 0), (3, 200, 300, 0), (2, 5, 0, 0), (2, 200, 0, 0),
                                       (50, 1, 0, 9000), (50, 1, 400, 0), (1, 600, 600, 600)])
@pytest.mark.parametrize("causal", [False, True])
def test_nothing_on_one_side(B, Sq, Sk, P, causal):
    run(B, Sq, Sk, P, 6, 2, 64, causal=causal, seed=3)


def test_no_queries():
    e = lambda n, c: torch.empty(n, c, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, lse = Q.attention_prefix(e(0, 128), e(6, 64), e(6, 64), e(9, 64), e(9, 64), 2, 1, 64, batch=2)
    assert o.shape == (0, 128) and lse.shape == (2, 2, 0)


def test_same_as_attention_over_both():
    s, o, lse = run(4, 200, 300, 500, 4, 2, 128, dtype="fp16", causal=True, seed=4)
    join = lambda p, x: torch.cat([torch.cat([p, x[b * 300:(b + 1) * 300]]) for b in range(4)])  # noqa: E731
    o1, lse1 = Q.attention(s["q"], join(s["pk"], s["k"]), join(s["pv"], s["v"]), 4, 2, 128, batch=4, causal=True)
    assert (o.float() - o1.float()).abs().max() < 2e-3 and (lse - lse1).abs().max() < 1e-5


def test_equal_calls_give_equal_bits_graph_and_streams():
    for shape in ((48, 1, 64, 3000), (3, 300, 200, 700)):
        s, o, lse = run(*shape, 8, 2, 128, seed=5)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            o2, lse2 = call(s, stream=side)
            side.synchronize()
            assert same_bits(o, o2) and same_bits(lse, lse2)
        lens, graph = torch.full((s["B"],), s["Sk"], dtype=torch.int32, device="cuda"), torch.cuda.CUDAGraph()
        args = (s["q"], s["k"], s["v"], s["pk"], s["pv"], 8, 2, 128)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            go, gl = Q.attention_prefix(*args, batch=s["B"], k_lens=lens)
        for n in (s["Sk"], 1, 0, 50):
            lens.fill_(n)
            graph.replay()
            eo, el = Q.attention_prefix(*args, batch=s["B"], k_lens=lens)
            torch.cuda.synchronize()
            assert same_bits(go, eo) and same_bits(gl, el)


def test_waits_are_bounded():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=Q.FLAG_TEST_STALL, wait_limit_ns=20_000_000, dev_status=word)
    for shape in ((48, 1, 64, 3000), (3, 300, 200, 700)):
        s = make(*shape, 8, 2, 128, seed=6)
        word.zero_()
        call(s, **kw)
        assert int(word.item()) == Q.ERR_TIMEOUT
        o, lse = call(s)
        check(s, o, lse)


@pytest.mark.parametrize("B,Sq,Sk,P,Hq,Hk,D", [
    (1, 4000, 4000, 130, 4, 4, 128),      # causal tiles as two halves, the prefix a small part
    (3, 1, 5000, 3000, 6, 2, 64),         # own keys long enough to be cut
    (3, 3, 5000, 200, 16, 1, 128),
    (24, 130, 64, 20000, 2, 2, 64),       # tiles of 256 rows in both passes
    (5, 16, 700, 9000, 3, 3, 128),
])
@pytest.mark.parametrize("causal", [False, True])
def test_each_way_through(B, Sq, Sk, P, Hq, Hk, D, causal):
    run(B, Sq, Sk, P, Hq, Hk, D, causal=causal, k_lens=None if B == 1 else [Sk - 7 * i for i in range(B)][:B] if Sk > 7 * B else None, seed=8)


def test_a_workspace_full_of_nan():
    # whatever a workspace held, every part that a join adds up has been written
    for shape, heads in (((64, 1, 100, 3000), (8, 2, 128)), ((3, 1, 5000, 3000), (6, 2, 64)), ((16, 40, 64, 4000), (6, 2, 128)),
                         ((2, 300, 300, 4000), (6, 6, 64))):
        s = make(*shape, *heads, k_lens=[(i * 37) % (shape[2] + 1) for i in range(shape[0])], seed=9)
        ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")
        o, lse = call(s, workspace=ws)
        o2, lse2 = call(s)
        assert same_bits(o, o2) and same_bits(lse, lse2)
        check(s, o, lse)


def test_outputs_beside_inputs():
    # q and o as columns of one buffer, keys of prefix and samples as columns of another
    s, o, lse = run(40, 2, 64, 3000, 4, 2, 64, seed=10)
    wide = torch.full((80, 2 * 256 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :256] = s["q"]
    far = dict(s, q=wide[:, :256])
    o2, _ = call(far, out=wide[:, 256:512])
    assert same_bits(o, o2) and same_bits(wide[:, :256], s["q"]) and (wide[:, 512:] == 7.0).all()
