"""More of what the training operators' C entry points refuse or work out
before any CUDA call.  Host only, with fake addresses, as in
test_training_abi_host."""
import ctypes

import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q
from tests.test_training_abi_host import FAKE, OVERLAP, changed, fake, lib, ln, refused  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only tests with fake device addresses")

LAST = (600 - 1) * 1536 * 2           # bytes to x's last row


@pytest.mark.parametrize("change", [
    dict(mean=FAKE), dict(rstd=FAKE + LAST + 1536 * 2 - 4),      # onto x: its first element, its last
    dict(mean=fake(2)), dict(rstd=fake(2) + 1536 * 4 - 4),       # onto the weight
    dict(mean=fake(3) + 4), dict(rstd=fake(3)),                  # onto the bias
    dict(rstd=fake(4)), dict(rstd=fake(4) + 599 * 4),            # onto each other
    dict(mean=FAKE + 64, y=None), dict(rstd=FAKE + 64, y=None),  # in place
])
def test_layer_norm_refuses_statistics_on_other_tensors(lib, change):  # noqa: F811
    refused(lib, "qknr_ln_forward", changed(ln, change), OVERLAP)
