"""Layer norm's backward pass where a CTA takes several units (chunks of one
sample's rows) one after the other.

With more than 4096 columns a CTA has a single group of warps and nothing
between its units but the row sums' own barriers, so units of an odd number
of steps are the ones to look at: the last step of a unit and the first of
the next must not share a buffer of sums.  Bounds as in test_layernorm_gpu."""
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from tests.test_layernorm_gpu import _lib, both  # noqa: F401  (the fixture)
from tests.training_util import same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,rpb", [(700, 1), (1001, 3), (1000, 7), (1830, 5), (900, 20)])
@pytest.mark.parametrize("C", [4104, 5120, 6144, 8192])
def test_samples_of_wide_rows(T, rpb, C):
    # one row each; odd numbers of rows; about as many samples as CTAs
    s, (_, mean, rstd), grads = both(T, C, "bf16", "act", rpb, True, seed=T + rpb + C)
    for _ in range(5):
        again = Q.layer_norm_backward(s["dy"], s["x"], s["weight"], mean, rstd, rows_per_batch=rpb, unit_offset=True)
        assert all(same_bits(a, b) for a, b in zip(again, grads))


@pytest.mark.parametrize("T,rpb", [(700, 1), (1001, 3), (1830, 5)])
@pytest.mark.parametrize("C", [3000, 4096])
def test_samples_of_two_groups(T, rpb, C):
    both(T, C, "fp16", "fp32", rpb, seed=T + rpb + C)


def test_one_row_of_any_stride():
    s, (y, mean, rstd), grads = both(1, 512, seed=3)
    wide = torch.zeros(1, 2 * 512 + 3, dtype=torch.bfloat16, device="cuda")
    x, dy = wide[:, :512], s["dy"].view(512, 1).clone().t()       # row strides of 1027 and of 1
    x.copy_(s["x"])
    assert x.stride(0) % 8 and dy.stride(0) == 1
    got = Q.layer_norm(x, s["weight"], s["bias"])
    got += Q.layer_norm_backward(dy, x, s["weight"], mean, rstd)
    assert all(same_bits(a, b) for a, b in zip(got, (y, mean, rstd, *grads)))
