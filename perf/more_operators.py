"""Workloads of the operators around attention over sequences of different
lengths: the root-mean-square norm with the residual's addition, its 8-bit
form and its gradients, attention of packed sequences with its backward pass,
and attention of a batch that shares a prefix of keys.

Every case is one pass through one operator, as a training or serving step
calls it.  ``run`` computes it in plain torch operations in 32 bits, or, where
``own`` is true, through the library's entry points; ``exact`` computes it in
64 bits from the definition.

Activations are token rows, [tokens, hidden] or [tokens, heads * head_dim].
Packed sequences follow each other without padding: sequence b is the rows
starts[b] .. starts[b + 1].
"""
import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
F8, F8_MAX, F8_SCALE_MIN = torch.float8_e4m3fn, 448.0, 2.0 ** -126


# ---------------------------------------------------------------------------
# the cases

def _rms(name, tokens, hidden, dtype="bf16", param="fp32", residual=True, samples=0, scales=""):
    """samples: 0 for one gain of all rows, else one (1 + scale) per sample;
    scales: "" for an output of the activations' type, "row" or "block" for 8
    bits with a scale per row or per 128 columns."""
    return {"name": name, "op": "rms_norm", "tokens": tokens, "hidden": hidden, "dtype": dtype, "param": param,
            "residual": residual, "samples": samples, "scales": scales}


def _rms_bwd(name, tokens, hidden, dtype="bf16", param="fp32", residual=True, samples=0):
    return {"name": name, "op": "rms_norm_backward", "tokens": tokens, "hidden": hidden, "dtype": dtype, "param": param,
            "residual": residual, "samples": samples}


def _packed(name, op, batch, seq_q, seq_k, heads_q, heads_k, head_dim, dtype="bf16", causal=False, lens=1):
    """seq_k 0: self-attention, keys packed like the queries.  The longest
    sequences have seq_q and seq_k tokens, the others by `lens`."""
    return {"name": name, "op": op, "batch": batch, "seq_q": seq_q, "seq_k": seq_k, "heads_q": heads_q, "heads_k": heads_k,
            "head_dim": head_dim, "dtype": dtype, "causal": causal, "lens": lens}


def _prefix(name, batch, seq_q, seq_k, prefix, heads_q, heads_k, head_dim, dtype="bf16", causal=False, lens=0):
    """lens 0: every sample has all its seq_k keys of its own."""
    return {"name": name, "op": "attention_prefix", "batch": batch, "seq_q": seq_q, "seq_k": seq_k, "prefix": prefix,
            "heads_q": heads_q, "heads_k": heads_k, "head_dim": head_dim, "dtype": dtype, "causal": causal, "lens": lens}


def listed():
    return [
        # the smallest norm call: a 256-token image, where latency counts
        _rms("rms_256x1536", 256, 1536),
        # the modulated norm between the two halves of a FLUX.2 block, 2 x (512 text + 4096 image) tokens, straight into
        # the 8-bit input of the projection behind it
        _rms("rms_fp8_2x4608x6144", 9216, 6144, param="bf16", samples=2, scales="row"),
        # a scale per 128 columns, an odd number of rows, fp16
        _rms("rms_fp8_block_1001x5120_fp16", 1001, 5120, dtype="fp16", scales="block"),
        # the gradients of the same block's norm, the residual stream's own gradient added
        _rms_bwd("rms_bwd_9216x6144", 9216, 6144),
        # and of a text encoder's on an odd number of rows, fp16, without a residual
        _rms_bwd("rms_bwd_1999x2048_fp16", 1999, 2048, dtype="fp16", residual=False),
        # a handful of short prompts through an autoregressive text encoder: latency
        _packed("packed_prompts_5x77x16x4x64", "attention_packed", 5, 77, 0, 16, 4, 64, causal=True, lens=3),
        # one pooling query over each of 16 images of different resolution: a single row per head
        _packed("packed_pool_16x1x4096x24x128", "attention_packed", 16, 1, 4096, 24, 24, 128, lens=5),
        # self-attention of a FLUX.2 block over images of different resolution in one batch
        _packed("packed_images_4x4608x48x128", "attention_packed", 4, 4608, 0, 48, 48, 128, lens=7),
        # gradient of a text encoder's layer over prompts of different lengths: causal, shared key heads, fp16
        _packed("packed_bwd_prompts_9x1999x16x4x64_fp16", "attention_packed_backward", 9, 1999, 0, 16, 4, 64, dtype="fp16",
                causal=True, lens=11),
        # gradient of the self-attention of images of different resolution
        _packed("packed_bwd_images_6x4096x24x128", "attention_packed_backward", 6, 4096, 0, 24, 24, 128, lens=13),
        # a token for each of 64 samples of one 8190-token prompt, each with up to 512 tokens of its own
        _prefix("prefix_token_64x1x512x8190x24x8x128", 64, 1, 512, 8190, 24, 8, 128, lens=17),
        # four images of 1024 tokens sampled beside one reference of 4608 tokens, FLUX.2's heads
        _prefix("prefix_images_4x1024x4608x48x128", 4, 1024, 1024, 4608, 48, 48, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_norm", "rms_norm", "rms_norm_backward", "attention_packed", "attention_packed_backward", "attention_prefix"])
    dtype = rng.choice(["bf16", "fp16"])
    lens = rng.randint(1, 1 << 20)
    if op.startswith("rms_norm"):
        scales = rng.choice(["", "row", "block"]) if op == "rms_norm" else ""
        hidden = 8 * _log_int(rng, 8, 1024) if scales != "block" else 128 * _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, min(16384, 9216 * 6144 // hidden))
        args = ("", tokens, hidden, dtype, rng.choice(["fp32", dtype]), rng.random() < 0.7, rng.choice([0, 0, 1, 2, 3]))
        c = _rms(*args, scales) if op == "rms_norm" else _rms_bwd(*args)
    else:
        heads_k, group, head_dim = rng.randint(1, 12), rng.choice([1, 1, 2, 4]), rng.choice([64, 128])
        heads = (heads_k * group, heads_k, head_dim, dtype, rng.random() < 0.5)
        if op == "attention_prefix":
            batch = _log_int(rng, 1, 64)
            seq_q = rng.choice([1, 1, rng.randint(2, 16), _log_int(rng, 17, 2048)])
            seq_q = max(1, min(seq_q, 4096 // batch))
            c = _prefix("", batch, seq_q, _log_int(rng, seq_q, 2048), _log_int(rng, 1, 8192), *heads, rng.choice([0, lens]))
        else:
            batch = _log_int(rng, 1, 32)
            seq_q = 1 if op == "attention_packed" and rng.random() < 0.25 else _log_int(rng, 1, min(4096, 16384 // batch))
            seq_k = 0 if seq_q > 1 and rng.random() < 0.7 else _log_int(rng, 1, min(4096, 32768 // batch))
            c = _packed("", op, batch, seq_q, seq_k, *heads, lens)
    del c["name"]
    return c


def _lengths(longest, batch, seed):
    """Tokens of each sequence: one is the longest, the others are shorter,
    of many one in eight empty.  Single tokens stay single."""
    if longest <= 1 or seed == 0:
        return [longest] * batch
    rng = random.Random(seed)
    lens = [0 if batch >= 8 and rng.random() < 0.125 else max(1, int(longest * rng.random())) for _ in range(batch)]
    lens[rng.randrange(batch)] = longest
    return lens


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _lens_q(case):
    return _lengths(case["seq_q"], case["batch"], case["lens"])


def _lens_k(case):
    return _lengths(case["seq_k"], case["batch"], case["lens"] + 1) if case["seq_k"] else _lens_q(case)


def _own_lens(case):
    return _lengths(case["seq_k"], case["batch"], case["lens"])


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype, scale=1.0, offset=0.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).add_(offset).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_rms(case, gen):
    tokens, hidden, dtype, param = case["tokens"], case["hidden"], DTYPES[case["dtype"]], DTYPES[case["param"]]
    per = -(-tokens // case["samples"]) if case["samples"] else None
    s = {"rows_per_batch": per}
    # a modulation is added to a gain of one; a learned gain stands by itself
    shape = (-(-tokens // per), hidden) if per else (hidden,)
    s["weight"] = _normal(gen, shape, param, 0.25, 0.0 if per else 1.0)
    s["x"] = _normal(gen, (tokens, hidden), dtype)
    if case["op"] == "rms_norm":
        s["residual"] = _normal(gen, (tokens, hidden), dtype, 2.0, 0.25) if case["residual"] else None
        return s
    # backward: x is the sum that the forward pass gave
    s["dy"] = _normal(gen, (tokens, hidden), dtype, 0.1)
    s["dsum"] = _normal(gen, (tokens, hidden), dtype, 0.1) if case["residual"] else None
    s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
    return s


def _prepare_packed(case, gen):
    hq, hk, d, dtype = case["heads_q"], case["heads_k"], case["head_dim"], DTYPES[case["dtype"]]
    lq, lk = _lens_q(case), _lens_k(case)
    rows_q, rows_k = sum(lq), sum(lk)
    s = {"q_starts": _int32(_starts(lq)), "lens": (lq, lk)}
    if not case["seq_k"]:
        qkv = _normal(gen, (rows_q, (hq + 2 * hk) * d), dtype)
        q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
        s["k_starts"] = s["q_starts"]
    else:
        q = _normal(gen, (rows_q, hq * d), dtype)
        kv = _normal(gen, (rows_k, 2 * hk * d), dtype)
        k, v = kv[:, :hk * d], kv[:, hk * d:]
        s["k_starts"] = _int32(_starts(lk))
    s.update(q=q, k=k, v=v)
    if case["op"] == "attention_packed_backward":
        s["do"] = _normal(gen, (rows_q, hq * d), dtype, 0.1)
        s["o"], s["lse"] = _plain_packed(case, s)
    return s


def _prepare_prefix(case, gen):
    batch, nq, nk, n, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "prefix", "heads_q", "heads_k", "head_dim"))
    dtype = DTYPES[case["dtype"]]
    q = _normal(gen, (batch * nq, hq * d), dtype)
    kv, shared = _normal(gen, (batch * nk, 2 * hk * d), dtype), _normal(gen, (n, 2 * hk * d), dtype)
    return {"q": q, "k": kv[:, :hk * d], "v": kv[:, hk * d:], "prefix_k": shared[:, :hk * d], "prefix_v": shared[:, hk * d:],
            "k_lens": _int32(_own_lens(case)) if case["lens"] else None}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = _prepare_rms if case["op"].startswith("rms") else _prepare_prefix if case["op"] == "attention_prefix" else _prepare_packed
    return {"case": case, **make(case, gen)}


# ---------------------------------------------------------------------------
# the plain forms

def _gain(case, s):
    """The gain of every row, [tokens, hidden] or [1, hidden]."""
    w = s["weight"].float()
    if not s["rows_per_batch"]:
        return w[None]
    return (1.0 + w)[torch.arange(case["tokens"], device="cuda") // s["rows_per_batch"]]


def _plain_rms(case, s):
    dtype = s["x"].dtype
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = h * rstd * _gain(case, s)
    out = [rstd.view(-1)] + ([h.to(dtype)] if s["residual"] is not None else [])
    if not case["scales"]:
        return [y.to(dtype)] + out
    blocks = y.view(case["tokens"], -1, 128 if case["scales"] == "block" else case["hidden"])
    scale = (blocks.abs().amax(2) / F8_MAX).clamp_min(F8_SCALE_MIN)
    values = (blocks / scale[..., None]).view(y.shape).to(F8)
    return [values, scale if case["scales"] == "block" else scale.view(-1)] + out


def _plain_rms_backward(case, s):
    h, dy = s["x"].float(), s["dy"].float()
    xhat = h * s["rstd"][:, None]
    g = dy * _gain(case, s)
    dx = s["rstd"][:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    terms = dy * xhat
    per = s["rows_per_batch"]
    if not per:
        return dx.to(s["x"].dtype), terms.sum(0)
    pad = s["weight"].shape[0] * per - case["tokens"]
    terms = torch.nn.functional.pad(terms, (0, 0, 0, pad)).view(-1, per, case["hidden"])
    return dx.to(s["x"].dtype), terms.sum(1)


def _spread(rows, starts, longest):
    """Packed rows as [batch, longest, columns] in 32 bits, and which of them are there."""
    at = torch.arange(longest, device="cuda")[None] + starts[:-1, None].long()
    there = at < starts[1:, None]
    return rows.float()[torch.where(there, at, 0)], there


def _split(t, heads, d):
    return t.view(t.shape[0], t.shape[1], heads, d).transpose(1, 2)


def _packed_scores(case, s):
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    longest_q, longest_k = max(s["lens"][0]), max(s["lens"][1])
    q, in_q = _spread(s["q"], s["q_starts"], longest_q)
    k, in_k = _spread(s["k"], s["k_starts"], longest_k)
    v, _ = _spread(s["v"], s["k_starts"], longest_k)
    # places past a sequence hold another row: none of it may count
    q, k, v = q * in_q[..., None], k * in_k[..., None], v * in_k[..., None]
    q, k, v = _split(q, hq, d), _split(k, hk, d).repeat_interleave(hq // hk, 1), _split(v, hk, d).repeat_interleave(hq // hk, 1)
    seen = in_q[:, None, :, None] & in_k[:, None, None, :]
    if case["causal"]:
        # the diagonal ends at the last query and the last key
        off = (s["k_starts"].diff() - s["q_starts"].diff())[:, None, None, None]
        i, j = torch.arange(longest_q, device="cuda")[:, None], torch.arange(longest_k, device="cuda")[None]
        seen = seen & (j <= i + off)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    return q, k, v, scores, in_q, in_k


def _softmax(scores):
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    return p, total, (top + total.log()).squeeze(3)


def _plain_packed(case, s):
    _, _, v, scores, in_q, _ = _packed_scores(case, s)
    p, total, lse = _softmax(scores)
    # a row that sees no key answers zero, and its log-sum is -inf
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return o.transpose(1, 2)[in_q].reshape(s["q"].shape).to(s["q"].dtype), lse.transpose(0, 1)[:, in_q].contiguous()


def _plain_packed_backward(case, s):
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    q, k, v, scores, in_q, in_k = _packed_scores(case, s)
    longest_q, longest_k, group = in_q.shape[1], in_k.shape[1], hq // hk
    do = _split(_spread(s["do"], s["q_starts"], longest_q)[0] * in_q[..., None], hq, d)
    o = _split(_spread(s["o"], s["q_starts"], longest_q)[0] * in_q[..., None], hq, d)
    lse = _spread(s["lse"].t(), s["q_starts"], longest_q)[0].transpose(1, 2)[..., None]
    p = scores.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_()
    delta = (do * o).sum(3, keepdim=True)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_(delta).mul_(p).mul_(1.0 / math.sqrt(d))
    dq = torch.matmul(ds, k)
    # the gradients of a shared key head are summed over its query heads
    dk = torch.matmul(ds.transpose(2, 3), q).view(-1, hk, group, longest_k, d).sum(2)
    dv = torch.matmul(p.transpose(2, 3), do).view(-1, hk, group, longest_k, d).sum(2)
    dtype = s["q"].dtype
    return (dq.transpose(1, 2)[in_q].reshape(s["q"].shape).to(dtype), dk.transpose(1, 2)[in_k].reshape(s["k"].shape).to(dtype),
            dv.transpose(1, 2)[in_k].reshape(s["v"].shape).to(dtype))


def _plain_prefix(case, s):
    batch, nq, nk, n, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "prefix", "heads_q", "heads_k", "head_dim"))
    group = hq // hk
    heads = lambda t, b, h: _split(t.float().reshape(b, -1, h * d), h, d)  # noqa: E731
    q = heads(s["q"], batch, hq)
    k, v = heads(s["k"], batch, hk).repeat_interleave(group, 1), heads(s["v"], batch, hk).repeat_interleave(group, 1)
    pk, pv = heads(s["prefix_k"], 1, hk).repeat_interleave(group, 1), heads(s["prefix_v"], 1, hk).repeat_interleave(group, 1)
    lens = torch.full((batch,), nk, device="cuda") if s["k_lens"] is None else s["k_lens"]
    j = torch.arange(nk, device="cuda")[None, None, None]
    seen = j < lens[:, None, None, None]
    if case["causal"]:
        seen = seen & (j <= torch.arange(nq, device="cuda")[None, None, :, None] + (lens - nq)[:, None, None, None])
    scores = torch.cat([torch.matmul(q, pk.transpose(2, 3)), torch.matmul(q, k.transpose(2, 3)).masked_fill_(~seen, -math.inf)], 3)
    p, total, lse = _softmax(scores.mul_(1.0 / math.sqrt(d)))
    o = (torch.matmul(p[..., :n], pv) + torch.matmul(p[..., n:], v)) / total
    return o.transpose(1, 2).reshape(s["q"].shape).to(s["q"].dtype), lse


def _plain(case, s):
    return {"rms_norm": _plain_rms, "rms_norm_backward": _plain_rms_backward, "attention_packed": _plain_packed,
            "attention_packed_backward": _plain_packed_backward, "attention_prefix": _plain_prefix}[case["op"]](case, s)


# ---------------------------------------------------------------------------
# the library's entry points

def _library(case, s):
    from diffusion_transformer_qk_gb300 import qknr as Q

    op = case["op"]
    if op.startswith("rms_norm"):
        kw = dict(rows_per_batch=s["rows_per_batch"], unit_offset=bool(s["rows_per_batch"]))
        if op == "rms_norm_backward":
            return Q.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dsum=s["dsum"], **kw)
        if not case["scales"]:
            y, rstd, h = Q.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, **kw)
            return [y, rstd] + ([h] if s["residual"] is not None else [])
        y, scale, rstd, h = Q.rms_norm_quantized(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                                                 block=128 if case["scales"] == "block" else None, **kw)
        return [y, scale, rstd] + ([h] if s["residual"] is not None else [])
    heads = (case["heads_q"], case["heads_k"], case["head_dim"])
    if op == "attention_packed":
        return Q.attention_packed(s["q"], s["k"], s["v"], *heads, s["q_starts"], s["k_starts"], causal=case["causal"])
    if op == "attention_packed_backward":
        return Q.attention_packed_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], *heads, s["q_starts"], s["k_starts"],
                                           causal=case["causal"])
    return Q.attention_prefix(s["q"], s["k"], s["v"], s["prefix_k"], s["prefix_v"], *heads, batch=case["batch"],
                              causal=case["causal"], k_lens=s["k_lens"])


def run(state):
    return list((_library if own else _plain)(state["case"], state))


# ---------------------------------------------------------------------------
# what a pass cannot do without

def _seen_pairs(nq, nk, causal):
    """Query-key pairs of one head of one sequence."""
    if not causal:
        return nq * nk
    # query i sees keys 0 .. i + nk - nq
    first = max(0, nq - nk)
    return (first + nk - nq + 1 + nk) * (nq - first) // 2 if nq > first else 0


def work(case):
    op = case["op"]
    if op.startswith("rms_norm"):
        n, rows = case["tokens"] * case["hidden"], case["tokens"]
        sets = max(1, case["samples"]) * case["hidden"]
        size = 4 if case["param"] == "fp32" else 2
        if op == "rms_norm_backward":
            return {"bytes": (8 if case["residual"] else 6) * n + sets * (size + 4) + 4 * rows, "flops": 10 * n}
        out = 2 * n if not case["scales"] else n + 4 * (rows if case["scales"] == "row" else n // 128)
        return {"bytes": (6 if case["residual"] else 2) * n + out + sets * size + 4 * rows, "flops": 6 * n}
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    if op == "attention_prefix":
        lens = _own_lens(case) if case["lens"] else [case["seq_k"]] * case["batch"]
        nq, nk = case["batch"] * case["seq_q"] * hq, (sum(lens) + case["prefix"]) * hk
        pairs = hq * sum(case["seq_q"] * case["prefix"] + _seen_pairs(case["seq_q"], n, case["causal"]) for n in lens)
        return {"bytes": 2 * d * (2 * nq + 2 * nk) + 4 * nq, "flops": 4 * d * pairs}
    lq, lk = _lens_q(case), _lens_k(case)
    pairs = hq * sum(_seen_pairs(a, b, case["causal"]) for a, b in zip(lq, lk))
    nq, nk = sum(lq) * hq, sum(lk) * hk
    if op == "attention_packed":
        return {"bytes": 2 * d * (2 * nq + 2 * nk) + 4 * nq, "flops": 4 * d * pairs}
    # q, o, do read and dq written; k, v read, dk and dv written
    return {"bytes": 2 * d * (4 * nq + 4 * nk) + 4 * nq, "flops": 10 * d * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_rms(case, s):
    tokens, hidden = case["tokens"], case["hidden"]
    per = s["rows_per_batch"] or tokens
    parts = []
    for b, first in enumerate(range(0, tokens, per)):
        rows = slice(first, min(tokens, first + per))
        w = (1.0 + s["weight"][b].double()) if s["rows_per_batch"] else s["weight"].double()
        h = s["x"][rows].double()
        if case["op"] == "rms_norm_backward":
            dy, r = s["dy"][rows].double(), s["rstd"][rows].double()[:, None]
            c = torch.einsum("rc,rc,c->r", dy, h, w)[:, None] / hidden
            dx = r * dy * w - h * r.pow(3) * c
            if s["dsum"] is not None:
                dx += s["dsum"][rows].double()
            parts.append([dx, torch.einsum("rc,rc,r->c", dy, h, r[:, 0])[None]])
            continue
        if s["residual"] is not None:
            h += s["residual"][rows].double()
        rms = torch.sqrt(torch.einsum("rc,rc->r", h, h) / hidden + EPS)
        y = h / rms[:, None] * w
        out = [1.0 / rms] + ([h] if s["residual"] is not None else [])
        if not case["scales"]:
            parts.append([y] + out)
            continue
        scales = []
        for c0 in range(0, hidden, 128 if case["scales"] == "block" else hidden):
            cols = y[:, c0:c0 + (128 if case["scales"] == "block" else hidden)]
            top = torch.maximum(cols.max(1).values, -cols.min(1).values)
            scales.append(torch.clamp(top / F8_MAX, min=F8_SCALE_MIN))
            cols /= scales[-1][:, None]
        parts.append([y, torch.stack(scales, 1) if case["scales"] == "block" else scales[0]] + out)
    got = [torch.cat(p) for p in zip(*parts)]
    if case["op"] == "rms_norm_backward" and not s["rows_per_batch"]:
        got[1] = got[1][0]
    return got


def _exact_packed(case, s):
    hq, hk, d = case["heads_q"], case["heads_k"], case["head_dim"]
    group, scale, back = hq // hk, 1.0 / math.sqrt(d), case["op"] == "attention_packed_backward"
    lq, lk = s["lens"]
    at_q, at_k = _starts(lq), _starts(lk)
    o = torch.zeros(sum(lq), hq * d, dtype=torch.float64, device="cuda")
    lse = torch.full((hq, sum(lq)), -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk = torch.zeros(sum(lk), hk * d, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    for b in range(case["batch"]):
        nq, nk = lq[b], lk[b]
        # queries from `first` on see a key
        first = max(0, nq - nk) if case["causal"] else 0
        if nk == 0 or first >= nq:
            continue
        rows, cols = slice(at_q[b] + first, at_q[b] + nq), slice(at_k[b], at_k[b] + nk)
        hidden = None
        if case["causal"]:
            hidden = torch.ones(nq - first, nk, dtype=torch.bool, device="cuda").triu(first + nk - nq + 1)
        for h in range(hq):
            hc, kc = slice(h * d, (h + 1) * d), slice(h // group * d, (h // group + 1) * d)
            q, k, v = s["q"][rows, hc].double(), s["k"][cols, kc].double(), s["v"][cols, kc].double()
            t = (q * scale) @ k.T
            if hidden is not None:
                t[hidden] = -math.inf
            if not back:
                lse[h, rows] = torch.logsumexp(t, 1)
                o[rows, hc] = torch.softmax(t, 1) @ v
                continue
            p = torch.exp(t - s["lse"][h, rows].double()[:, None])
            do = s["do"][rows, hc].double()
            dv[cols, kc] += p.T @ do
            ds = p * (do @ v.T - torch.einsum("rd,rd->r", do, s["o"][rows, hc].double())[:, None])
            dq[rows, hc] = ds @ (k * scale)
            dk[cols, kc] += ds.T @ (q * scale)
    return [dq, dk, dv] if back else [o, lse]


def _exact_prefix(case, s):
    batch, nq, nk, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "heads_q", "heads_k", "head_dim"))
    group, scale = hq // hk, 1.0 / math.sqrt(d)
    lens = _own_lens(case) if case["lens"] else [nk] * batch
    o = torch.zeros(batch * nq, hq * d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(batch, hq, nq, dtype=torch.float64, device="cuda")
    for h in range(hq):
        hc, kc = slice(h * d, (h + 1) * d), slice(h // group * d, (h // group + 1) * d)
        pk, pv = s["prefix_k"][:, kc].double(), s["prefix_v"][:, kc].double()
        for b, n in enumerate(lens):
            rows, cols = slice(b * nq, (b + 1) * nq), slice(b * nk, b * nk + n)
            q = s["q"][rows, hc].double() * scale
            t = q @ s["k"][cols, kc].double().T
            if case["causal"]:
                # query i sees keys 0 .. i + n - nq
                t[torch.ones(nq, n, dtype=torch.bool, device="cuda").triu(n - nq + 1)] = -math.inf
            t = torch.cat([q @ pk.T, t], 1)
            lse[b, h] = torch.logsumexp(t, 1)
            o[rows, hc] = torch.softmax(t, 1) @ torch.cat([pv, s["v"][cols, kc].double()])
    return [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rms_norm"):
        return _exact_rms(case, s)
    return _exact_prefix(case, s) if case["op"] == "attention_prefix" else _exact_packed(case, s)
