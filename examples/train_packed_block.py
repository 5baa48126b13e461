"""Training steps of an autoregressive block over packed prompts of different
lengths, on one GPU:

    y   = rms_norm(x, g1)
    qkv = qk_norm_rope(y @ w_qkv)                     positions begin anew in every prompt
    a   = attention_packed(q, k, v, starts) @ w_out   causal, each prompt by itself
    h   = x + a,  z = rms_norm(h, g2)                 one call
    out = h + z @ w_up

and its backward pass, with the framework's kernels for everything but the
projections; and a sampling step of several samples that share one prompt
(``sample``), whose norms give the projections' inputs in 8 bits.

    python examples/train_packed_block.py [--steps N] [--prompts B] [--tokens S]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from diffusion_transformer_qk_gb300 import qknr as Q  # noqa: E402

TRAINED = ("w_qkv", "w_out", "w_up", "gamma_q", "gamma_k", "g1", "g2")


def tables(positions, dim):
    """cos and sin of the rotation at each position, [rows, dim]."""
    freq = torch.exp(-math.log(10000.0) * torch.arange(0, dim, 2, device="cuda") / dim)
    angle = (positions[:, None] * freq).repeat_interleave(2, dim=1)
    return angle.cos().contiguous(), angle.sin().contiguous()


class PackedBlock:
    """``params`` holds TRAINED: the projections in the activation dtype, the
    gains in float32."""

    def __init__(self, params, heads_q, heads_k, dim):
        self.p, self.heads_q, self.heads_k, self.dim = params, heads_q, heads_k, dim
        self.heads = (heads_q, heads_k, dim)

    def _columns(self, packed):
        return packed.split([h * self.dim for h in (self.heads_q, self.heads_k, self.heads_k)], dim=1)

    def forward(self, x, starts, cos, sin):
        """x: the prompts' token rows, one after the other; ``starts`` int32
        [prompts + 1].  Returns the output and what backward() needs."""
        p = self.p
        y, rstd1, _ = Q.rms_norm(x, p["g1"])
        qkv = y @ p["w_qkv"]
        normed = Q.qk_norm_rope_packed(qkv, self.heads_q, self.heads_k, self.heads_k, self.dim, p["gamma_q"], p["gamma_k"],
                                       cos, sin, out=torch.empty_like(qkv))
        o, lse = Q.attention_packed(*self._columns(normed), *self.heads, starts, causal=True)
        z, rstd2, h = Q.rms_norm(o @ p["w_out"], p["g2"], residual=x)
        return torch.addmm(h, z, p["w_up"]), (x, y, rstd1, qkv, normed, o, lse, h, z, rstd2)

    def backward(self, dout, kept, starts, cos, sin):
        """Gradients of x and of the parameters."""
        x, y, rstd1, qkv, normed, o, lse, h, z, rstd2 = kept
        p = self.p
        g = {"w_up": z.t() @ dout}
        da, g["g2"] = Q.rms_norm_backward(dout @ p["w_up"].t(), h, p["g2"], rstd2, dsum=dout)
        g["w_out"] = o.t() @ da
        d = torch.empty_like(qkv)                # gradients of q, k, v side by side
        dq, dk, dv = self._columns(d)
        Q.attention_packed_backward(da @ p["w_out"].t(), *self._columns(normed), o, lse, *self.heads, starts, causal=True, dq=dq,
                                    dk=dk, dv=dv)
        _, g["gamma_q"], g["gamma_k"] = Q.qk_norm_rope_packed_backward(
            d, qkv, self.heads_q, self.heads_k, self.heads_k, self.dim, p["gamma_q"], p["gamma_k"], cos, sin)   # in place
        g["w_qkv"] = y.t() @ d
        dx, g["g1"] = Q.rms_norm_backward(d @ p["w_qkv"].t(), x, p["g1"], rstd1, dsum=da, out=da)
        return dx, g

    def keys(self, x, cos, sin):
        """The keys and values of one prompt's rows, normalised and rotated."""
        y, _, _ = Q.rms_norm(x, self.p["g1"])
        qkv = y @ self.p["w_qkv"]
        Q.qk_norm_rope_packed(qkv, self.heads_q, self.heads_k, self.heads_k, self.dim, self.p["gamma_q"], self.p["gamma_k"], cos, sin)
        return self._columns(qkv)[1:]

    def sample(self, x, prefix_k, prefix_v, cache_k, cache_v, lens, cos, sin):
        """One token for each of several samples of a prompt: x [batch, C], the
        prompt's keys and values, the samples' own in cache_k and cache_v
        [batch * most, Hk * D], ``lens`` int32 [batch] of them so far (the new
        token's go behind them).  The norms' outputs are 8 bits with a scale."""
        p, batch = self.p, x.shape[0]
        y, scale, _, _ = Q.rms_norm_quantized(x, p["g1"])
        qkv = (y.to(x.dtype) * scale[:, None].to(x.dtype)) @ p["w_qkv"]
        Q.qk_norm_rope_packed(qkv, self.heads_q, self.heads_k, self.heads_k, self.dim, p["gamma_q"], p["gamma_k"], cos, sin)
        q, k, v = self._columns(qkv)
        at = torch.arange(batch, device=x.device) * (cache_k.shape[0] // batch) + lens
        cache_k[at], cache_v[at] = k, v
        o, _ = Q.attention_prefix(q, cache_k, cache_v, prefix_k, prefix_v, *self.heads, batch=batch, k_lens=lens + 1)
        z, scale, _, h = Q.rms_norm_quantized(o @ p["w_out"], p["g2"], residual=x)
        return torch.addmm(h, z.to(x.dtype) * scale[:, None].to(x.dtype), p["w_up"])


def make_block(lens, heads_q, heads_k, dim, dtype=torch.bfloat16, seed=0):
    """A block with random weights, the prompts' starts and tables, one batch."""
    gen = torch.Generator("cuda").manual_seed(seed)
    C, rows = heads_q * dim, sum(lens)

    def normal(*shape, scale=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    params = {"w_qkv": normal(C, (heads_q + 2 * heads_k) * dim, scale=C ** -0.5, dt=dtype),
              "w_out": normal(C, C, scale=C ** -0.5, dt=dtype), "w_up": normal(C, C, scale=C ** -0.5, dt=dtype),
              "gamma_q": 1 + normal(dim, scale=0.1), "gamma_k": 1 + normal(dim, scale=0.1),
              "g1": 1 + normal(C, scale=0.1), "g2": 1 + normal(C, scale=0.1)}
    starts = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    positions = torch.cat([torch.arange(n, device="cuda") for n in lens])
    x, target = normal(rows, C, dt=dtype), normal(rows, C, dt=dtype)
    return PackedBlock(params, heads_q, heads_k, dim), x, target, starts, *tables(positions, dim)


def step(block, x, target, starts, cos, sin, rate):
    """One step of gradient descent on mean((out - target)^2); returns the loss."""
    out, kept = block.forward(x, starts, cos, sin)
    diff = out.float() - target.float()
    _, grads = block.backward((diff * (2.0 / diff.numel())).to(x.dtype), kept, starts, cos, sin)
    for name in TRAINED:
        block.p[name] -= (rate * grads[name].float()).to(block.p[name].dtype)
    return (diff * diff).mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prompts", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=1024, help="of the longest prompt")
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--key-heads", type=int, default=4)
    ap.add_argument("--head-dim", type=int, default=64)
    args = ap.parse_args(argv)
    lens = [max(1, args.tokens * (args.prompts - b) // args.prompts) for b in range(args.prompts)]
    block, *data = make_block(lens, args.heads, args.key_heads, args.head_dim)
    rate = 0.02 * data[0].numel() ** 0.5         # the gradients shrink with the loss's mean
    losses = [step(block, *data, rate) for _ in range(3)]
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    losses += [step(block, *data, rate) for _ in range(args.steps)]
    end.record()
    torch.cuda.synchronize()
    if Q.read_status():
        raise RuntimeError("a kernel reported an error")
    print(f"loss {losses[0].item():.4f} -> {losses[-1].item():.4f}, {start.elapsed_time(end) / max(args.steps, 1):.3f} ms per step")
    return [loss.item() for loss in losses]


if __name__ == "__main__":
    main()
