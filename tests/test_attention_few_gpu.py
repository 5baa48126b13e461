"""Attention of a few queries over many keys (one token of decoding, a pooling
token), with the bounds of tests/test_attention_gpu.py: shared heads, masks,
key lengths around the ends of the warps' steps, results split over CTAs."""
import pytest
import torch

import tests.test_attention_gpu as TA
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.training_util import same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0


# (queries, query heads, key heads): 1 to 16 queries, up to 16 rows of a key head and more; 17 for the other kernel
@pytest.mark.parametrize("Sq,Hq,Hk", [(1, 1, 1), (1, 3, 3), (1, 4, 2), (1, 3, 1), (1, 8, 2), (2, 3, 3), (2, 4, 2), (3, 2, 2),
                                      (4, 1, 1), (1, 5, 1), (1, 18, 2), (8, 2, 2), (5, 3, 1), (16, 2, 2), (1, 20, 1), (16, 6, 2), (7, 5, 1), (17, 1, 1)])
@pytest.mark.parametrize("Sk", [1, 2, 7, 8, 9, 63, 128, 129, 255, 257, 384, 511, 1000])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_sizes(Sq, Hq, Hk, Sk, D, dtype):
    TA.both(2, Sq, Sk, Hq, Hk, D, dtype=dtype, seed=Sk + Sq)


@pytest.mark.parametrize("Sq,Sk,Hq,Hk", [(1, 5000, 1, 1), (4, 3001, 1, 1), (1, 2999, 4, 1), (2, 2000, 2, 1), (11, 3003, 2, 2), (9, 2500, 4, 1)])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_keys_shared_out_over_many_ctas(Sq, Sk, Hq, Hk, D, dtype):
    TA.both(1, Sq, Sk, Hq, Hk, D, dtype=dtype, seed=3)


@pytest.mark.parametrize("batch,heads", [(160, 1), (100, 4), (51, 7)])
def test_more_heads_than_ctas(batch, heads):
    TA.both(batch, 1, 600, heads, heads, 64, seed=4)


@pytest.mark.parametrize("Sq,Sk", [(1, 300), (3, 300), (4, 2), (4, 1), (3, 1500), (16, 300), (13, 5)])
def test_causal(Sq, Sk):
    TA.both(2, Sq, Sk, 2, 2, 64, causal=True, seed=5)


@pytest.mark.parametrize("q_lens,k_lens", [([1, 0, 1, 1], [0, 700, 1, 300]), ([0, 0, 0, 0], None), (None, [0, 0, 0, 0]),
                                           (None, [5, 600, 128, 8])])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(2, 2), (4, 1)])
def test_lengths_with_nan_behind_them(q_lens, k_lens, causal, Hq, Hk):
    TA.both(4, 1, 700, Hq, Hk, 128, causal=causal, q_lens=q_lens, k_lens=k_lens, seed=6)


def test_more_queries_with_lengths():
    TA.both(3, 4, 600, 1, 1, 64, q_lens=[4, 2, 0], k_lens=[600, 1, 77], causal=True, seed=7)


@pytest.mark.parametrize("size", [0.01, 8.0])
def test_flat_and_peaked_rows(size):
    TA.both(2, 1, 3000, 2, 2, 128, size=size, seed=8)


def test_packed_columns_and_equal_bits():
    s = TA.make(3, 4, 4, 2, 2, 64, packed=True, seed=9)
    o, lse = TA.forward(s)
    TA.check_forward(s, "bf16", o, lse)
    again = TA.forward(s)
    assert same_bits(o, again[0]) and same_bits(lse, again[1])
    big = TA.make(8, 1, 4096, 6, 6, 128, seed=10)
    one, two = TA.forward(big), TA.forward(big)
    assert all(same_bits(a, b) for a, b in zip(one, two))


def test_decoding_a_sequence_matches_the_causal_pass():
    """Token by token over a growing cache: the cache is one buffer, its valid
    keys a length on the device, and one captured graph serves every token."""
    S, Hq, Hk, D = 70, 4, 2, 64
    s = TA.make(1, S, S, Hq, Hk, D, causal=True, seed=11)
    whole, _ = TA.forward(s)
    q = torch.empty_like(s["q"][:1])
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    step = lambda: Q.attention(q, s["k"], s["v"], Hq, Hk, D, k_lens=n)
    for _ in range(2):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = step()
    for t in range(S):
        q.copy_(s["q"][t:t + 1])
        n.fill_(t + 1)
        graph.replay()
        # two kernels' roundings of the same row: a bf16 step of the values, at most 4
        assert (o.float() - whole[t:t + 1].float()).abs().max().item() <= 4 * torch.finfo(torch.bfloat16).eps, t


def test_a_wait_that_runs_out_is_reported():
    s = TA.make(2, 1, 3000, 4, 2, 64, seed=16)
    o, lse = TA.forward(s)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    TA.forward(s, flags=Q.FLAG_TEST_STALL, wait_limit_ns=2_000_000, dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == Q.ERR_TIMEOUT
    # the context is whole: the next call is right
    assert same_bits(TA.forward(s)[0], o)


def test_checked_build(libs_checked):
    TA.both(2, 1, 1000, 4, 2, 128, seed=12)
    TA.both(1, 3, 5000, 1, 1, 64, causal=True, seed=13)
    TA.both(160, 1, 300, 2, 2, 64, seed=14)
    TA.both(1, 12, 3000, 1, 1, 128, seed=15)


@pytest.fixture
def libs_checked(built_lib, monkeypatch):
    from diffusion_transformer_qk_gb300 import build as B
    monkeypatch.setattr(Q, "_lib", Q.load(B.ensure_built(checked=True)))
    monkeypatch.setattr(Q, "_plans", {})
    yield
    torch.cuda.synchronize()
    assert Q.read_status() == 0
