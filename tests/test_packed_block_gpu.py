"""The operators of sequences together: the block of
examples/train_packed_block.py against the same block written with torch's own
operators, prompt by prompt, in 64 bits and in the activation dtype.

Bound.  As for the attention block: both 16-bit forms round the same
intermediates, so the framework's error against 64 bits may be twice the plain
form's, plus the rounding of the result itself."""
import importlib.util
import os

import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "train_packed_block",
    os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_packed_block.py"))
E = importlib.util.module_from_spec(spec)
spec.loader.exec_module(E)


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0


def rms(t, gain):
    return t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * gain


def plain(block, x, dout, starts, cos, sin, dtype):
    """The block with torch's operators and its autograd."""
    Hq, Hk, D = block.heads
    small = lambda t: t.detach().to(dtype).requires_grad_()  # noqa: E731
    p = {n: small(t) for n, t in block.p.items()}
    x = small(x)
    qkv = (rms(x, p["g1"]) @ p["w_qkv"]).view(-1, Hq + 2 * Hk, D)

    def prepare(t, gamma):
        t = rms(t, gamma)
        turned = torch.stack((-t[..., 1::2], t[..., 0::2]), -1).flatten(-2)
        return t * cos.to(dtype)[:, None] + turned * sin.to(dtype)[:, None]

    q, k, v = prepare(qkv[:, :Hq], p["gamma_q"]), prepare(qkv[:, Hq:Hq + Hk], p["gamma_k"]), qkv[:, Hq + Hk:]
    k, v = k.repeat_interleave(Hq // Hk, 1), v.repeat_interleave(Hq // Hk, 1)
    rows = []
    at = starts.tolist()
    for a, b in zip(at, at[1:]):
        s = torch.einsum("ihd,jhd->hij", q[a:b], k[a:b]) * D ** -0.5
        s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        rows.append(torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v[a:b]))
    h = x + torch.cat(rows).reshape(x.shape[0], Hq * D) @ p["w_out"]
    out = h + rms(h, p["g2"]) @ p["w_up"]
    grads = torch.autograd.grad(out, [x] + [p[n] for n in E.TRAINED], dout.to(dtype))
    return [out.detach(), *grads]


@pytest.mark.parametrize("lens,Hq,Hk,D,dtype", [([77, 300, 20, 129], 4, 2, 64, torch.bfloat16), ([256, 400], 3, 1, 128, torch.bfloat16),
                                                ([31, 0, 200, 77, 128], 2, 2, 64, torch.float16)])
def test_block_matches_plain(lens, Hq, Hk, D, dtype):
    block, x, dout, starts, cos, sin = E.make_block(lens, Hq, Hk, D, dtype, seed=sum(lens))
    out, kept = block.forward(x, starts, cos, sin)
    dx, g = block.backward(dout, kept, starts, cos, sin)
    got = [out, dx] + [g[n] for n in E.TRAINED]
    exact = plain(block, x, dout, starts, cos, sin, torch.float64)
    rounded = plain(block, x, dout, starts, cos, sin, dtype)
    for name, a, e, r in zip(("out", "x") + E.TRAINED, got, exact, rounded):
        size = e.norm().item()
        own, theirs = (a.double() - e).norm().item(), (r.double() - e).norm().item()
        assert own <= 2 * theirs + torch.finfo(dtype).eps / 2 * size, (name, own / size, theirs / size)


def test_gradients_against_differences():
    # the loss along each parameter's own gradient, in steps that stand clear of 16-bit noise: the slope is |g|^2
    # (10 %: the quadratic terms of three layers' products over a step of 2 %)
    block, x, dout, starts, cos, sin = E.make_block([120, 64, 200], 4, 2, 64, torch.float16, seed=1)
    out, kept = block.forward(x, starts, cos, sin)
    _, g = block.backward(dout, kept, starts, cos, sin)
    loss = lambda: (block.forward(x, starts, cos, sin)[0].double() * dout.double()).sum().item()  # noqa: E731
    for name in E.TRAINED:
        old, way = block.p[name], g[name].double()
        size = 0.02 * old.double().norm() / way.norm()
        ends, moves = [], []
        for sign in (1, -1):
            block.p[name] = (old.double() + sign * size * way).to(old.dtype)
            moves.append(((block.p[name].double() - old.double()) * way).sum().item())
            ends.append(loss())
        block.p[name] = old
        slope = (ends[0] - ends[1]) / (moves[0] - moves[1])
        assert abs(slope - 1) < 0.1, (name, slope)


def test_the_example_runs():
    losses = E.main(["--steps", "3", "--prompts", "4", "--tokens", "200", "--heads", "4", "--key-heads", "2"])
    assert all(l == l and l < 1e3 for l in losses)


def test_a_step_in_a_graph_gives_the_eager_bits():
    block, x, dout, starts, cos, sin = E.make_block([150, 300, 40], 4, 2, 64, seed=5)
    for _ in range(2):
        out, kept = block.forward(x, starts, cos, sin)
        dx, g = block.backward(dout, kept, starts, cos, sin)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.backward(dout, block.forward(x, starts, cos, sin)[1], starts, cos, sin)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2, kept2 = block.forward(x, starts, cos, sin)
        dx2, g2 = block.backward(dout, kept2, starts, cos, sin)
    for t in (out2, dx2, *g2.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(dx, dx2)
    for n in E.TRAINED:
        assert torch.equal(g[n], g2[n]), n


@pytest.mark.parametrize("batch,prompt", [(3, 200), (40, 3000)])
def test_sampling_continues_the_prompt(batch, prompt):
    """Tokens sampled beside the shared prompt: each sample's rows are those
    of a packed sequence prompt + own tokens, but for the norms' 8 bits.

    Bound: e4m3 rounds each of the two norms' values by at most 2^-4 of
    itself (2^-5.3 in the mean square for values spread evenly between powers
    of two), independently over the C values a projection adds up, so the
    projections' results move by less than 2^-4 of their size, and the block's
    output, h plus such a projection, by less than 2^-3 of its own."""
    Hq, Hk, D, steps = 4, 2, 64, 3
    block, x, _, _, cos, sin = E.make_block([prompt] + [steps] * batch, Hq, Hk, D, seed=7)
    pk, pv = block.keys(x[:prompt], cos[:prompt].contiguous(), sin[:prompt].contiguous())
    own = x[prompt:].view(batch, steps, -1)
    caches = [torch.zeros(batch * 8, Hk * D, dtype=x.dtype, device="cuda") for _ in range(2)]
    got = []
    for s in range(steps):
        lens = torch.full((batch,), s, dtype=torch.int32, device="cuda")
        c, sn = E.tables(torch.full((batch,), prompt + s, device="cuda"), D)
        got.append(block.sample(own[:, s].contiguous(), pk, pv, *caches, lens, c, sn))
    c, sn = E.tables(torch.arange(prompt + steps, device="cuda"), D)
    starts = torch.tensor([0, prompt + steps], dtype=torch.int32, device="cuda")
    for b in (0, batch // 2, batch - 1):
        rows = torch.cat([x[:prompt], own[b]])
        ref = block.forward(rows, starts, c, sn)[0][prompt:].double()
        mine = torch.stack([got[s][b] for s in range(steps)]).double()
        assert (mine - ref).norm() <= 2.0 ** -3 * ref.norm()
