"""Shared helpers of the training operators' GPU tests."""
import numpy as np
import torch

from tests.gpu_util import TORCH

U = 2.0 ** -24                       # half a step of fp32, relative


def half_step(dtype: str) -> float:
    """Largest relative error of one rounding into the type."""
    return torch.finfo(TORCH[dtype]).eps / 2


def smallest(dtype: str) -> float:
    """Half a step among the type's subnormals: the error of a rounding near zero."""
    return {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}[dtype]


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def normal(gen, shape, dtype, scale=1.0, offset=0.0):
    x = torch.from_numpy(gen.normal(size=shape) * scale + offset)
    return x.to(dtype).cuda()


def within(got, ref, bound, what=""):
    """|got - ref| <= bound, element by element."""
    got = f64(got).reshape(ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    over = np.abs(got - ref) - bound
    worst = int(np.argmax(over)) if over.size else 0
    assert over.size == 0 or over.flat[worst] <= 0, \
        f"{what}: {got.flat[worst]} against {ref.flat[worst]}, bound {np.broadcast_to(bound, ref.shape).flat[worst]}"


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
