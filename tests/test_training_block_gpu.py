"""The training operators together: the attention block of
examples/train_attention_block.py against the same block written with torch's
own operators, in 64 bits and in the activation dtype.

Bound.  Both 16-bit forms round the same intermediates (y, qkv, the
normalised qkv, p, o, and their gradients), so their errors against 64 bits
are samples of one size; the framework's may be twice the plain form's, plus
the rounding of the result itself.  That holds where the gradients are not
zero by cancellation, so not for a single token, whose q and k have none (that
case is among the attention's own sizes, with a bound of its own)."""
import importlib.util
import os

import pytest
import torch

from diffusion_transformer_qk_gb300 import qknr as Q

pytestmark = pytest.mark.gpu

spec = importlib.util.spec_from_file_location(
    "train_attention_block",
    os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_attention_block.py"))
E = importlib.util.module_from_spec(spec)
spec.loader.exec_module(E)


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0


def plain(block, x, dout, dtype):
    """The block with torch's operators and its autograd."""
    B, H, D = block.batch, block.heads, block.dim
    S, C = x.shape[0] // B, x.shape[1]
    small = lambda t: t.detach().to(dtype).requires_grad_()
    p = {n: small(t) for n, t in block.p.items()}
    x = small(x)
    xs = x.view(B, S, C)
    y = torch.nn.functional.layer_norm(xs, (C,), eps=1e-6) * (1 + p["scale"][:, None]) + p["shift"][:, None]
    qkv = (y.view(B * S, C) @ p["w_qkv"]).view(B, S, 3, H, D)

    def prepare(t, gamma):
        t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + 1e-6) * gamma
        turned = torch.stack((-t[..., 1::2], t[..., 0::2]), -1).flatten(-2)
        return (t * block.cos.to(dtype)[:, None] + turned * block.sin.to(dtype)[:, None]).transpose(1, 2)

    q, k, v = prepare(qkv[:, :, 0], p["gamma_q"]), prepare(qkv[:, :, 1], p["gamma_k"]), qkv[:, :, 2].transpose(1, 2)
    o = torch.softmax(q @ k.transpose(2, 3) * D ** -0.5, -1) @ v
    out = x + o.transpose(1, 2).reshape(B * S, C) @ p["w_out"]
    grads = torch.autograd.grad(out, [x] + [p[n] for n in E.TRAINED], dout.to(dtype))
    return [out.detach(), *grads]


@pytest.mark.parametrize("B,S,H,D,dtype", [(2, 256, 4, 64, torch.bfloat16), (1, 300, 3, 128, torch.bfloat16),
                                           (3, 77, 2, 64, torch.float16)])
def test_block_matches_plain(B, S, H, D, dtype):
    block, x, dout = E.make_block(B, S, H, D, dtype, seed=S)
    out, kept = block.forward(x)
    dx, g = block.backward(dout, kept)
    got = [out, dx] + [g[n] for n in E.TRAINED]
    exact, rounded = plain(block, x, dout, torch.float64), plain(block, x, dout, dtype)
    for name, a, e, r in zip(("out", "x") + E.TRAINED, got, exact, rounded):
        size = e.norm().item()
        own, theirs = (a.double() - e).norm().item(), (r.double() - e).norm().item()
        assert own <= 2 * theirs + torch.finfo(dtype).eps / 2 * size, (name, own / size, theirs / size)


def test_the_example_learns():
    losses = E.main(["--steps", "10", "--tokens", "256", "--heads", "4"])
    assert losses[-1] < losses[0]


def test_a_step_in_a_graph_gives_the_eager_bits():
    block, x, dout = E.make_block(2, 200, 3, 64, seed=5)
    for _ in range(2):
        out, kept = block.forward(x)
        dx, g = block.backward(dout, kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.backward(dout, block.forward(x)[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out2, kept2 = block.forward(x)
        dx2, g2 = block.backward(dout, kept2)
    for t in (out2, dx2, *g2.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(dx, dx2)
    for n in E.TRAINED:
        assert torch.equal(g[n], g2[n]), n
