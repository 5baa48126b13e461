"""Packed attention and attention beside a shared prefix where the plan cuts
tiles of long sequences beside many short ones: against the fp64 oracle, on a
workspace that held NaN."""
import numpy as np
import pytest
import torch

import tests.test_attention_packed_gpu as P
import tests.test_attention_prefix_gpu as X
from diffusion_transformer_qk_gb300 import qknr as Q
from tests.gpu_util import TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


@pytest.fixture(scope="module")
def workspace(cuda_device):
    return torch.empty(1 << 28, dtype=torch.uint8, device="cuda")


def run(s, workspace, backward=True):
    td = TORCH[s["dtype"]]
    o, lse = P.kept(*s["q"].shape, dtype=td), P.kept(s["Hq"], s["q"].shape[0])
    P.call(s, out=o, lse=lse, workspace=workspace.fill_(255))
    P.check_forward(s, o, lse)
    if backward:
        grads = [P.kept(*t.shape, dtype=td) for t in (s["q"], s["k"], s["v"])]
        P.call_backward(s, s["do"], o, lse, dq=grads[0], dk=grads[1], dv=grads[2], workspace=workspace.fill_(255))
        P.check_backward(s, o, lse, *grads)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,Hq,Hk", [([1000] * 39 + [640] * 63, 4, 2), ([640] * 63 + [1000] * 39, 2, 2)])
def test_a_query_each(lens, Hq, Hk, dtype, D, workspace):
    run(P.make([1] * len(lens), lens, Hq, Hk, D, dtype=dtype, seed=51), workspace, backward=D == 64)


@pytest.mark.parametrize("seed", range(16))
def test_a_few_queries_each_at_random(seed, workspace):
    gen = np.random.Generator(np.random.PCG64(200 + seed))
    B = int(gen.integers(33, 201))
    if seed % 2:
        lens = gen.integers(500, 4001, size=B)
    else:
        lens = np.where(gen.random(B) < gen.random(), int(gen.integers(900, 4001)), int(gen.integers(100, 901)))
    Hk, group, D = int(gen.integers(1, 5)), int(gen.choice([1, 3, 8])), int(gen.choice([64, 128]))
    rows = [1] * B if seed % 4 < 2 else gen.integers(0, 4, size=B).tolist()
    run(P.make(rows, lens.tolist(), Hk * group, Hk, D, dtype="fp16" if seed & 4 else "bf16", causal=bool(seed & 8), seed=seed), workspace,
        backward=False)


@pytest.mark.parametrize("lens,H,causal", [([3000] * 3 + [512] * 33, 3, False), ([3375] * 2 + [512] * 28, 2, False),
                                           ([512] * 28 + [3375] * 2, 2, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_long_prompts_beside_short_ones(lens, H, causal, dtype, workspace):
    run(P.make(lens, None, H, H, 64, dtype=dtype, causal=causal, seed=52), workspace)


@pytest.mark.parametrize("seed", range(6))
def test_prompts_at_random(seed, workspace):
    gen = np.random.Generator(np.random.PCG64(300 + seed))
    lens = [int(gen.integers(1800, 3400))] * int(gen.integers(1, 3)) + [int(gen.choice([300, 384, 512, 640]))] * int(gen.integers(10, 35))
    Hk, group = int(gen.integers(1, 3)), int(gen.choice([1, 2]))
    run(P.make(gen.permutation(lens).tolist(), None, Hk * group, Hk, 128 if seed == 5 else 64, causal=bool(seed & 1),
               dtype="fp16" if seed & 2 else "bf16", seed=seed), workspace)


def prefix(s, workspace):
    X.check(s, *X.call(s, workspace=workspace.fill_(255)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P_", [700, 6000])
def test_own_keys_of_two_lengths(P_, D, workspace):
    prefix(X.make(64, 1, 1152, P_, 16, 4, D, k_lens=[640] * 20 + [1152] + [640] * 43, seed=53), workspace)


@pytest.mark.parametrize("seed", range(8))
def test_own_keys_at_random(seed, workspace):
    gen = np.random.Generator(np.random.PCG64(400 + seed))
    B, Sk = int(gen.integers(33, 65)), int(gen.integers(1025, 3000))
    k_lens = (gen.integers(0, Sk + 1, size=B) if seed % 2 else np.where(gen.random(B) < 0.2, Sk, int(gen.integers(300, 900)))).tolist()
    Hk, group, D = int(gen.integers(1, 5)), int(gen.choice([1, 4])), int(gen.choice([64, 128]))
    prefix(X.make(B, int(gen.integers(1, 4)), Sk, int(gen.integers(200, 5000)), Hk * group, Hk, D, dtype="fp16" if seed & 4 else "bf16",
                  k_lens=k_lens, causal=bool(seed & 2), seed=seed), workspace)
