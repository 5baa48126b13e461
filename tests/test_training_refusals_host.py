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


@pytest.mark.parametrize("T,C", [(600, 1536), (1000, 5120), (7, 64), (100, 9000)])
@pytest.mark.parametrize("rpb", [1 << 40, (1 << 63) - 600, (1 << 63) - 1])
def test_a_sample_longer_than_the_call_is_one_sample(lib, T, C, rpb):  # noqa: F811
    # however long: T + rows_per_batch need not fit in 64 bits
    sizes = []
    for value in (0, rpb):
        n = ctypes.c_size_t(7)
        assert lib.qknr_ln_workspace_bytes(ctypes.byref(changed(lambda: ln(T, C), dict(rows_per_batch=value))), ctypes.byref(n)) == 0
        sizes.append(n.value)
    assert sizes[0] == sizes[1]
