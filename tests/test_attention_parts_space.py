"""A packed call of a few queries whose shares may cut a tile (equal stretches of
the line, csrc/attn_kernel.cuh's table_span, restated in
test_attention_shares) has room for the parts in its workspace."""
import ctypes

import numpy as np
import pytest

from diffusion_transformer_qk_gb300 import qknr as Q
from tests.test_attention_shares import CTAS, blocks, even_spans, share_cut  # noqa: F401  (share_cut: the fixture)


@pytest.fixture(scope="module")
def lib(built_lib):
    return Q.load()


def workspace(lib, batch, rows_q, rows_k, Hq, Hk, D):
    a, n = Q.QknrPackArgs(), ctypes.c_size_t(0)
    lib.qknr_pack_args_init(ctypes.byref(a))
    a.batch, a.rows_q, a.rows_k, a.n_heads_q, a.n_heads_k, a.head_dim = batch, rows_q, rows_k, Hq, Hk, D
    assert lib.qknr_pack_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == Q.OK
    return n.value


def check(lib, cut, lens_q, lens_k, Hq, Hk, D, extra=0):
    group, batch = Hq // Hk, len(lens_q)
    tile = 8 if group * sum(lens_q) <= 8 * batch else 16
    line = np.array([blocks(k) + 4 for q, k in zip(lens_q, lens_k) for _ in range(-(-group * q // tile))], dtype=np.int64)
    space = workspace(lib, batch, sum(lens_q), sum(lens_k) + extra, Hq, Hk, D)
    if space == 0 or not line.size:               # tiles in waves, none of them cut
        return False
    cuts = any(u > 0 for _, u in even_spans(cut, line, Hk, 4, 4))
    if cuts:
        assert space >= 2 * CTAS * tile * (D * 4 + 8), (lens_q, lens_k, Hq, Hk, D)
    return cuts


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens_q,lens_k,Hq,Hk", [([1] * 20, [900] + [5] * 19, 16, 16), ([1] * 32, [512] * 2 + [0] * 30, 12, 12),
                                                 ([0] * 30 + [1, 1], [0] * 30 + [900, 100], 20, 20), ([1] * 12, [385] + [50] * 11, 96, 48)])
def test_short_keys_of_many_heads(lib, share_cut, lens_q, lens_k, Hq, Hk, D):  # noqa: F811
    assert check(lib, share_cut, lens_q, lens_k, Hq, Hk, D)


def test_at_random(lib, share_cut):  # noqa: F811
    n = 0
    for seed in range(1500):
        gen = np.random.Generator(np.random.PCG64(seed))
        B, Hk, group = int(gen.integers(1, 33)), int(gen.integers(1, 49)), int(gen.choice([1, 2, 4]))
        most = int(gen.choice([300, 1000, 1300, 4000]))
        lens_q = np.minimum(gen.integers(0, 17, size=B), int(gen.choice([1, 2, 16]))).tolist()
        lens_k = np.diff(np.sort(np.concatenate([[0, most], gen.integers(0, most + 1, size=B - 1)]))).tolist()
        if seed % 3 == 0:                         # one that has most of them
            lens_k = [most * 9 // 10] + [most // 10 // max(B - 1, 1)] * (B - 1)
        if not any(lens_q):
            continue
        n += check(lib, share_cut, lens_q, lens_k, Hk * group, Hk, int(gen.choice([64, 128])), extra=int(gen.choice([0, 0, 40])))
    assert n > 200
