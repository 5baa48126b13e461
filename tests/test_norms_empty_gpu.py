"""The norms' gradients of a batch without rows: the sum over nothing is zero,
whether or not the call says how many rows share a weight row."""
import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()


def tensors(n, C=256, dtype=torch.bfloat16):
    e = lambda *shape, t=torch.float32: torch.empty(*shape, dtype=t, device="cuda")  # noqa: E731
    return e(n, C, t=dtype), e(n, C, t=dtype), e(n), e(n)


@pytest.mark.parametrize("rpb", [None, 1, 5])
@pytest.mark.parametrize("given", [False, True])
def test_one_weight_row(rpb, given):
    x, dy, mean, rstd = tensors(0)
    weight = torch.ones(256, device="cuda")
    out = [torch.full((256,), 7.0, device="cuda") for _ in range(3)]
    if not given:                                 # the memory that a new tensor gets
        del out
    kw = dict(dweight=out[0], dbias=out[1]) if given else {}
    dx, dw, db = Q.layer_norm_backward(dy, x, weight, mean, rstd, rows_per_batch=rpb, **kw)
    assert dx.shape == (0, 256) and dw.shape == db.shape == (256,)
    dx, dg = Q.rms_norm_backward(dy, x, weight, rstd, rows_per_batch=rpb, **(dict(dweight=out[2]) if given else {}))
    assert dx.shape == (0, 256) and dg.shape == (256,)
    assert not any(t.any() for t in (dw, db, dg))


def test_a_row_for_each_sample():
    x, dy, mean, rstd = tensors(0)
    weight = torch.ones(3, 256, device="cuda")
    assert Q.layer_norm_backward(dy, x, weight, mean, rstd, rows_per_batch=5)[1].shape == (0, 256)
    assert Q.rms_norm_backward(dy, x, weight, rstd, rows_per_batch=5)[1].shape == (0, 256)
