"""Rows with one large score and very many small ones: each small probability
is below what a half holds beside the largest, all of them together are not.

Bound, with one key of score 0 and value a, N of score c and value w (so the
answer is (a + N w e^c) / (1 + N e^c)): a probability enters its product
rounded, by h of itself or, near zero, by 2^-25 2^-7 of the row's largest; the
sums over N + 1 keys, the scores and the output's rounding are as in
test_attention_gpu."""
import math

import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from tests.gpu_util import TORCH
from tests.training_util import U, f64, half_step, smallest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("a,w", [(0.0, 1.0), (1.0, -3.0)])
@pytest.mark.parametrize("Sq,H,N", [(256, 152, 65535), (300, 1, 65535), (1, 1, 65535), (16, 1, 131071)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_small_probabilities(dtype, D, Sq, H, N, a, w, first):
    td = TORCH[dtype]
    c = -17.75                                    # e^c = 2^-25.6; c / 4 is exact in both types
    q = torch.zeros((Sq, H * D), dtype=td, device="cuda")   # 152 heads: as many tiles as SMs, so that one takes all keys
    k = torch.zeros((N + 1, D), dtype=td, device="cuda")
    v = torch.full((N + 1, D), w, dtype=td, device="cuda")
    q[:, ::D], k[:, 0] = 4.0, c / 4
    at = 0 if first else N
    k[at], v[at] = 0, a
    o, lse = Q.attention(q, k, v, H, 1, D, scale=1.0)
    tail = N * math.exp(c)
    want, size = (a + w * tail) / (1 + tail), (abs(a) + abs(w) * tail) / (1 + tail)
    h, e = half_step(dtype), 2 * ((2 * D + 4) * U * abs(c) + 2.0 ** -22) + (2 * N + 18) * U
    near = 2.0 ** -32 if dtype == "fp16" else 2.0 ** -126
    bound = h * abs(want) + (h + e) * size + (N + 1) * near * max(abs(a), abs(w)) + smallest(dtype)
    assert float((o.double() - want).abs().max()) <= bound
    assert float((lse.double() - math.log1p(tail)).abs().max()) <= 2.0 ** -22 + e + 8 * U
