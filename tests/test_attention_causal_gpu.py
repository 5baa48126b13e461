"""Causal attention at sizes where its tiles go out in different ways: fewer
tiles than CTAs, cut in halves or in equal shares; about as many; several
waves; key heads shared by many query heads.  The bounds are those of
tests/test_attention_gpu.py."""
import pytest

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


@pytest.mark.parametrize("B,S,Hq,Hk,D", [(1, 1000, 2, 2, 64), (1, 2500, 3, 3, 128), (1, 2500, 6, 6, 64), (13, 1500, 1, 1, 64),
                                         (2, 1300, 16, 8, 64), (10, 2000, 4, 1, 64), (1, 640, 40, 40, 128)])
def test_sizes(B, S, Hq, Hk, D):
    TA.both(B, S, S, Hq, Hk, D, causal=True, seed=S + Hq)


def test_halves_of_many_blocks_on_shared_heads():
    # 11 tiles of each of 15 samples' key head, each up to 88 blocks
    TA.both(15, 1400, 1400, 8, 1, 64, causal=True, seed=41)


@pytest.mark.parametrize("q_lens,k_lens", [([2000, 1, 0, 777], None), (None, [2000, 130, 0, 1])])
def test_lengths(q_lens, k_lens):
    TA.both(4, 2000, 2000, 4, 2, 64, causal=True, q_lens=q_lens, k_lens=k_lens, seed=42)


def test_more_keys_than_queries_and_the_other_way_round():
    TA.both(1, 600, 3000, 3, 3, 128, causal=True, seed=43)
    TA.both(1, 3000, 600, 3, 3, 64, causal=True, seed=44)


def test_equal_calls_give_equal_bits():
    s = TA.make(1, 2500, 2500, 4, 4, 128, causal=True, seed=45)
    o, lse = TA.forward(s)
    grads = TA.backward(s, o, lse)
    again = TA.forward(s)
    assert all(same_bits(a, b) for a, b in zip((o, lse, *grads), (*again, *TA.backward(s, *again))))
