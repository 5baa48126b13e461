"""A few queries whose last key head is cut among all CTAs: 153 tiles, one
more than there are CTAs, leave each of them a handful of keys."""
import pytest

from tests.test_attention_gpu import _lib, check_forward, forward, make  # noqa: F401  (_lib: the fixture)
from tests.training_util import same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,Sq,Sk,Hq,Hk", [(9, 1, 1024, 17, 17), (9, 1, 1500, 34, 17), (9, 5, 1031, 51, 17), (17, 16, 2047, 9, 9),
                                           (17, 3, 1024, 144, 18)])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_one_tile_too_many(B, Sq, Sk, Hq, Hk, D, dtype):
    s = make(B, Sq, Sk, Hq, Hk, D, dtype, seed=Sk + Hq)
    o, lse = forward(s)
    check_forward(s, dtype, o, lse)
    assert all(same_bits(a, b) for a, b in zip(forward(s), (o, lse)))
    s = make(B, Sq, Sk, Hq, Hk, D, dtype, seed=Sk, causal=True, k_lens=[Sk - 100 * b for b in range(B)] if Sk > 100 * B else None)
    check_forward(s, dtype, *forward(s))
