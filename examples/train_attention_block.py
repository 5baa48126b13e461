"""Training steps of a diffusion transformer's attention block on one GPU:

    y   = layer_norm(x) * (1 + scale) + shift         modulated per sample
    qkv = y @ w_qkv
    qkv = qk_norm_rope(qkv)                           q, k normalised and rotated
    out = x + attention(q, k, v) @ w_out

and its backward pass, with the framework's kernels for everything but the
two projections.  The block keeps what the backward pass reads: y, mean and
rstd of the norm, qkv before and after the QK norm, o and lse of the
attention.

    python examples/train_attention_block.py [--steps N] [--batch B] [--tokens S]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from diffusion_transformer_qk_gb300 import qknr as Q  # noqa: E402

TRAINED = ("w_qkv", "w_out", "gamma_q", "gamma_k", "scale", "shift")


class AttentionBlock:
    """``params`` holds TRAINED: the projections in the activation dtype, the
    gains of Q and K [D] and the modulation [B, C] in float32."""

    def __init__(self, params, cos, sin, batch, n_heads, head_dim):
        self.p, self.cos, self.sin = params, cos, sin
        self.batch, self.heads, self.dim = batch, n_heads, head_dim

    def _columns(self, packed):
        return packed.split(self.heads * self.dim, dim=1)

    def forward(self, x):
        """x: token rows [B * S, C].  Returns the output and what backward() needs."""
        p, H, D = self.p, self.heads, self.dim
        rows = x.shape[0] // self.batch
        y, mean, rstd = Q.layer_norm(x, p["scale"], p["shift"], rows_per_batch=rows, unit_offset=True)
        qkv = y @ p["w_qkv"]
        # out of place: the backward pass needs the inputs
        normed = Q.qk_norm_rope_packed(qkv, H, H, H, D, p["gamma_q"], p["gamma_k"], self.cos, self.sin, cos_rows=rows,
                                       out=torch.empty_like(qkv))
        o, lse = Q.attention(*self._columns(normed), H, H, D, batch=self.batch)
        return torch.addmm(x, o, p["w_out"]), (x, y, mean, rstd, qkv, normed, o, lse)

    def backward(self, dout, kept):
        """Gradients of x and of the parameters."""
        x, y, mean, rstd, qkv, normed, o, lse = kept
        p, H, D = self.p, self.heads, self.dim
        rows = x.shape[0] // self.batch
        g = {"w_out": o.t() @ dout}
        do = dout @ p["w_out"].t()
        d = torch.empty_like(qkv)                # gradients of q, k, v side by side
        dq, dk, dv = self._columns(d)
        Q.attention_backward(do, *self._columns(normed), o, lse, H, H, D, batch=self.batch, dq=dq, dk=dk, dv=dv)
        _, g["gamma_q"], g["gamma_k"] = Q.qk_norm_rope_packed_backward(
            d, qkv, H, H, H, D, p["gamma_q"], p["gamma_k"], self.cos, self.sin, cos_rows=rows)      # in place
        g["w_qkv"] = y.t() @ d
        dx, g["scale"], g["shift"] = Q.layer_norm_backward(d @ p["w_qkv"].t(), x, p["scale"], mean, rstd, rows_per_batch=rows,
                                                           unit_offset=True)
        return dx.add_(dout), g


def make_block(batch, tokens, n_heads, head_dim, dtype=torch.bfloat16, seed=0):
    """A block with random weights, its rotation tables and one batch of data."""
    gen = torch.Generator("cuda").manual_seed(seed)
    C = n_heads * head_dim

    def normal(*shape, scale=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dt)

    params = {"w_qkv": normal(C, 3 * C, scale=C ** -0.5, dt=dtype), "w_out": normal(C, C, scale=C ** -0.5, dt=dtype),
              "gamma_q": 1 + normal(head_dim, scale=0.1), "gamma_k": 1 + normal(head_dim, scale=0.1),
              "scale": normal(batch, C, scale=0.1), "shift": normal(batch, C, scale=0.1)}
    freq = torch.exp(-math.log(10000.0) * torch.arange(0, head_dim, 2, device="cuda") / head_dim)
    angle = (torch.arange(tokens, device="cuda")[:, None] * freq).repeat_interleave(2, dim=1)
    x, target = normal(batch * tokens, C, dt=dtype), normal(batch * tokens, C, dt=dtype)
    return AttentionBlock(params, angle.cos().contiguous(), angle.sin().contiguous(), batch, n_heads, head_dim), x, target


def step(block, x, target, rate):
    """One step of gradient descent on mean((out - target)^2); returns the loss."""
    out, kept = block.forward(x)
    diff = out.float() - target.float()
    _, grads = block.backward((diff * (2.0 / diff.numel())).to(x.dtype), kept)
    for name in TRAINED:
        block.p[name] -= (rate * grads[name].float()).to(block.p[name].dtype)
    return (diff * diff).mean()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=24)
    ap.add_argument("--head-dim", type=int, default=64)
    args = ap.parse_args(argv)
    block, x, target = make_block(args.batch, args.tokens, args.heads, args.head_dim)
    rate = 0.02 * x.numel() ** 0.5               # the gradients shrink with the loss's mean
    losses = []
    for _ in range(3):
        losses.append(step(block, x, target, rate))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(args.steps):
        losses.append(step(block, x, target, rate))
    end.record()
    torch.cuda.synchronize()
    if Q.read_status():
        raise RuntimeError("a kernel reported an error")
    print(f"loss {losses[0].item():.4f} -> {losses[-1].item():.4f}, {start.elapsed_time(end) / max(args.steps, 1):.3f} ms per step")
    return [loss.item() for loss in losses]


if __name__ == "__main__":
    main()
