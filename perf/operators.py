"""Workloads of the training operators: layer norm with its gradients, the
backward pass of the fused QK-RMSNorm + RoPE, and attention with its backward
pass.

Every case is one pass through one operator, as a training (or sampling) step
of a diffusion transformer calls it.  ``run`` computes it in plain torch
operations in 32 bits, or, where ``own`` is true, through the library's entry
points; ``exact`` computes it in 64 bits from the definition.

Activations are token rows, [batch * seq, heads * head_dim] or
[batch * seq, hidden]; self-attention and the QK-norm gradient take column
views of one packed [tokens, (Hq + Hk + Hv) * head_dim] buffer.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# the cases

def _ln(name, op, batch, seq, hidden, dtype="bf16", param="fp32", modulated=False):
    return {"name": name, "op": op, "batch": batch, "seq": seq, "hidden": hidden, "dtype": dtype, "param": param,
            "modulated": modulated}


def _qk(name, batch, seq, heads_q, heads_k, head_dim, style, dtype="bf16", table="fp32"):
    return {"name": name, "op": "qk_norm_rope_backward", "batch": batch, "seq": seq, "heads_q": heads_q,
            "heads_k": heads_k, "head_dim": head_dim, "style": style, "dtype": dtype, "table": table}


def _attn(name, op, batch, seq_q, seq_k, heads_q, heads_k, head_dim, dtype="bf16", causal=False, ragged=False):
    return {"name": name, "op": op, "batch": batch, "seq_q": seq_q, "seq_k": seq_k, "heads_q": heads_q,
            "heads_k": heads_k, "head_dim": head_dim, "dtype": dtype, "causal": causal, "ragged": ragged}


def listed():
    return [
        # the smallest norm call: the final norm of a 256-token image, where latency counts
        _ln("ln_256x1536", "layer_norm", 1, 256, 1536),
        # the modulated norm before each attention of a FLUX.2 block: 2 x (512 text + 4096 image) tokens
        _ln("ln_mod_2x4608x6144", "layer_norm", 2, 4608, 6144, param="bf16", modulated=True),
        # its gradients, the scale and shift summed over each sample's rows
        _ln("ln_mod_bwd_2x4608x6144", "layer_norm_backward", 2, 4608, 6144, param="bf16", modulated=True),
        # an affine norm (cross-attention's query norm) on an odd number of rows, fp16
        _ln("ln_bwd_1001x5120_fp16", "layer_norm_backward", 1, 1001, 5120, dtype="fp16"),
        # QK-norm gradient of the 256-token workload: latency
        _qk("qk_bwd_256x24x64", 1, 256, 24, 24, 64, "interleaved"),
        # and of a FLUX.2 block
        _qk("qk_bwd_2x4608x48x128", 2, 4608, 48, 48, 128, "rotate_half"),
        # self-attention of the 256-token workload: latency
        _attn("attn_256x24x64", "attention", 1, 256, 256, 24, 24, 64),
        # one pooling query over each image's 4096 latent tokens: a single row per head
        _attn("attn_pool_8x1x4096x24x128", "attention", 8, 1, 4096, 24, 24, 128),
        # self-attention of a FLUX.2 block
        _attn("attn_2x4608x48x128", "attention", 2, 4608, 4608, 48, 48, 128),
        # gradient of Wan's cross-attention: two clips of a quarter of its 32760 latent tokens against up to 512 text
        # tokens (the second prompt is shorter)
        _attn("attn_cross_bwd_2x8190x512x40x128", "attention_backward", 2, 8190, 512, 40, 40, 128, ragged=True),
        # backward of a dense 4096-token self-attention
        _attn("attn_bwd_4096x24x128", "attention_backward", 1, 4096, 4096, 24, 24, 128),
        # causal, shared key heads, odd length, fp16: an autoregressive text encoder's layer
        _attn("attn_bwd_causal_3x1999x16x4x64_fp16", "attention_backward", 3, 1999, 1999, 16, 4, 64, dtype="fp16",
              causal=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "qk_norm_rope_backward", "attention", "attention_backward"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("layer_norm"):
        batch, hidden = rng.randint(1, 4), 8 * _log_int(rng, 8, 1024)
        c = _ln("", op, batch, _log_int(rng, 1, max(1, min(16384, 9216 * 6144 // hidden) // batch)), hidden, dtype,
                rng.choice(["fp32", dtype]), rng.random() < 0.5)
    elif op == "qk_norm_rope_backward":
        batch, heads_k, group, head_dim = rng.randint(1, 2), rng.randint(1, 24), rng.choice([1, 1, 2]), rng.choice([64, 128])
        c = _qk("", batch, _log_int(rng, 1, 4608), heads_k * group, heads_k, head_dim,
                rng.choice(["interleaved", "rotate_half"]), dtype, rng.choice(["fp32", "bf16"]))
    else:
        batch, heads_k, group, head_dim = rng.randint(1, 4), rng.randint(1, 12), rng.choice([1, 1, 2, 4]), rng.choice([64, 128])
        seq_q = _log_int(rng, 1, 4096 // batch)
        seq_k = seq_q if rng.random() < 0.5 else _log_int(rng, 1, 4096 // batch)
        c = _attn("", op, batch, seq_q, seq_k, heads_k * group, heads_k, head_dim, dtype, rng.random() < 0.3,
                  rng.random() < 0.4)
    del c["name"]
    return c


def _lengths(case):
    """Valid key tokens of each sample: all of them, or, where the batch is
    ragged, prompts of falling length, the last of four or more empty."""
    n, batch = case["seq_k"], case["batch"]
    if not case["ragged"]:
        return [n] * batch
    lens = [n - (3 * b * n) // (4 * batch) for b in range(batch)]
    if batch >= 4:
        lens[-1] = 0
    return lens


# ---------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype, scale=1.0, offset=0.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).add_(offset).to(dtype)


def _prepare_ln(case, gen):
    rows, hidden, dtype = case["batch"] * case["seq"], case["hidden"], DTYPES[case["dtype"]]
    sets, param = case["batch"] if case["modulated"] else 1, DTYPES[case["param"]]
    s = {"x": _normal(gen, (rows, hidden), dtype, 2.0, 0.25)}
    # a modulation is added to a gain of one; a learned gain stands by itself
    s["weight"] = _normal(gen, (sets, hidden), param, 0.25, 0.0 if case["modulated"] else 1.0)
    s["bias"] = _normal(gen, (sets, hidden), param, 0.25)
    if case["op"] == "layer_norm_backward":
        s["dy"] = _normal(gen, (rows, hidden), dtype, 0.1)
        x = s["x"].float()
        mean = x.mean(1)
        s["mean"], s["rstd"] = mean, ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()
    return s


def _prepare_qk(case, gen):
    batch, seq, d, dtype = case["batch"], case["seq"], case["head_dim"], DTYPES[case["dtype"]]
    rows, width = batch * seq, (case["heads_q"] + 2 * case["heads_k"]) * d
    # 1-D positions, base 10000; the table holds one row per position, shared by the batch
    angle = torch.arange(seq, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    angle = torch.cat([angle, angle], 1) if case["style"] == "rotate_half" else angle.repeat_interleave(2, 1)
    table = DTYPES[case["table"]]
    return {"qkv": _normal(gen, (rows, width), dtype, 2.0), "dout": _normal(gen, (rows, width), dtype, 0.1),
            "gamma_q": _normal(gen, (d,), torch.float32, 0.1, 1.0), "gamma_k": _normal(gen, (d,), torch.float32, 0.1, 1.0),
            "cos": angle.cos().to(table).contiguous(), "sin": angle.sin().to(table).contiguous()}


def _prepare_attn(case, gen):
    batch, nq, nk, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "heads_q", "heads_k", "head_dim"))
    dtype = DTYPES[case["dtype"]]
    if nq == nk:
        # normalised and rotated Q and K beside V in one packed buffer
        qkv = _normal(gen, (batch * nq, (hq + 2 * hk) * d), dtype)
        q, k, v = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
    else:
        q = _normal(gen, (batch * nq, hq * d), dtype)
        kv = _normal(gen, (batch * nk, 2 * hk * d), dtype)
        k, v = kv[:, :hk * d], kv[:, hk * d:]
    s = {"q": q, "k": k, "v": v,
         "k_lens": torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None}
    if case["op"] == "attention_backward":
        s["do"] = _normal(gen, (batch * nq, hq * d), dtype, 0.1)
        s["o"], s["lse"] = _plain_attention(case, s)
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    make = _prepare_ln if op.startswith("layer_norm") else _prepare_qk if op == "qk_norm_rope_backward" else _prepare_attn
    return {"case": case, **make(case, gen)}


# ---------------------------------------------------------------------------
# the plain forms

def _per_sample(case, rows):
    """Token rows [batch * seq, C] with the sample as an axis of its own."""
    sets = case["batch"] if case["modulated"] else 1
    return rows.float().view(sets, -1, rows.shape[1])


def _gain(case, s):
    w = s["weight"].float()
    return (1.0 + w if case["modulated"] else w)[:, None]


def _plain_layer_norm(case, s):
    x = _per_sample(case, s["x"])
    mean = x.mean(2, keepdim=True)
    d = x - mean
    rstd = (d.square().mean(2, keepdim=True) + EPS).rsqrt()
    y = d * rstd * _gain(case, s) + s["bias"].float()[:, None]
    return y.view(s["x"].shape).to(s["x"].dtype), mean.view(-1), rstd.view(-1)


def _plain_layer_norm_backward(case, s):
    x, dy = _per_sample(case, s["x"]), _per_sample(case, s["dy"])
    rstd = s["rstd"].view(x.shape[0], -1, 1)
    xhat = (x - s["mean"].view(x.shape[0], -1, 1)) * rstd
    g = dy * _gain(case, s)
    dx = rstd * (g - g.mean(2, keepdim=True) - xhat * (g * xhat).mean(2, keepdim=True))
    return dx.view(s["x"].shape).to(s["x"].dtype), (dy * xhat).sum(1), dy.sum(1)


def _partner(style, x):
    """x[..., p(d)], p(d) the rotation partner of dimension d."""
    if style == "rotate_half":
        return torch.cat([x[..., x.shape[-1] // 2:], x[..., :x.shape[-1] // 2]], -1)
    return x.view(*x.shape[:-1], -1, 2).flip(-1).reshape(x.shape)


def _sign(style, d):
    """s(d): -1 for the first member of a pair, +1 for the second."""
    one = torch.ones(d // 2, device="cuda")
    return torch.cat([-one, one]) if style == "rotate_half" else torch.stack([-one, one], 1).view(-1)


def _plain_qk_tensor(case, x, dout, gamma, s):
    style, d = case["style"], case["head_dim"]
    shape = (case["batch"], case["seq"], -1, d)
    x, do = x.float().reshape(shape), dout.float().reshape(shape)
    cos, sin = s["cos"].float()[:, None], s["sin"].float()[:, None]
    # y[d] reaches o[d] by cos[d] and o[p] by s(p) sin[p]
    dy = do * cos + _partner(style, do * sin * _sign(style, d))
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    g = dy * gamma
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx.reshape(case["batch"] * case["seq"], -1), (dy * x * r).sum((0, 1, 2))


def _plain_qk_backward(case, s):
    d, hq, hk = case["head_dim"], case["heads_q"], case["heads_k"]
    q0, k0 = hq * d, (hq + hk) * d
    dq, dgq = _plain_qk_tensor(case, s["qkv"][:, :q0], s["dout"][:, :q0], s["gamma_q"], s)
    dk, dgk = _plain_qk_tensor(case, s["qkv"][:, q0:k0], s["dout"][:, q0:k0], s["gamma_k"], s)
    return torch.cat([dq.to(s["qkv"].dtype), dk.to(s["qkv"].dtype), s["dout"][:, k0:]], 1), dgq, dgk


def _heads(case, t, n, heads):
    return t.float().reshape(case["batch"], n, heads, case["head_dim"]).transpose(1, 2)


def _visible(case, s):
    """[batch, 1, seq_q, seq_k]: which keys a query sees.  The causal diagonal
    ends at the last query and the sample's last valid key."""
    nq, nk = case["seq_q"], case["seq_k"]
    col = torch.arange(nk, device="cuda")[None, None, None, :]
    lens = torch.full((case["batch"],), nk, device="cuda") if s["k_lens"] is None else s["k_lens"].long()
    lens = lens[:, None, None, None]
    seen = (col < lens).expand(-1, -1, nq, -1)
    if case["causal"]:
        seen = seen & (col <= torch.arange(nq, device="cuda")[None, None, :, None] + lens - nq)
    return seen


def _scores(case, s, masked):
    group = case["heads_q"] // case["heads_k"]
    q = _heads(case, s["q"], case["seq_q"], case["heads_q"])
    k = _heads(case, s["k"], case["seq_k"], case["heads_k"]).repeat_interleave(group, 1)
    v = _heads(case, s["v"], case["seq_k"], case["heads_k"]).repeat_interleave(group, 1)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(case["head_dim"]))
    if case["causal"] or case["ragged"]:
        scores.masked_fill_(~_visible(case, s), masked)
    return q, k, v, scores


def _rows(case, t):
    return t.transpose(1, 2).reshape(case["batch"] * t.shape[2], -1)


def _plain_attention(case, s):
    _, _, v, scores = _scores(case, s, -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    # a row that sees no key answers zero, and its log-sum is -inf
    o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
    return _rows(case, o).to(s["q"].dtype), (top + total.log()).squeeze(3)


def _plain_attention_backward(case, s):
    batch, nk, hq, hk, d = (case[k] for k in ("batch", "seq_k", "heads_q", "heads_k", "head_dim"))
    q, k, v, scores = _scores(case, s, -math.inf)
    lse = s["lse"][..., None]
    p = scores.sub_(torch.where(lse == -math.inf, torch.zeros_like(lse), lse)).exp_()
    do = _heads(case, s["do"], case["seq_q"], hq)
    o = _heads(case, s["o"], case["seq_q"], hq)
    delta = (do * o).sum(3, keepdim=True)
    ds = torch.matmul(do, v.transpose(2, 3)).sub_(delta).mul_(p).mul_(1.0 / math.sqrt(d))
    dq = torch.matmul(ds, k)
    # the gradients of a shared key head are summed over its query heads
    dk = torch.matmul(ds.transpose(2, 3), q).view(batch, hk, -1, nk, d).sum(2)
    dv = torch.matmul(p.transpose(2, 3), do).view(batch, hk, -1, nk, d).sum(2)
    return [_rows(case, t).to(s["q"].dtype) for t in (dq, dk, dv)]


def _plain(case, s):
    op = case["op"]
    if op == "layer_norm":
        return _plain_layer_norm(case, s)
    if op == "layer_norm_backward":
        return _plain_layer_norm_backward(case, s)
    if op == "qk_norm_rope_backward":
        return _plain_qk_backward(case, s)
    if op == "attention":
        return _plain_attention(case, s)
    return _plain_attention_backward(case, s)


# ---------------------------------------------------------------------------
# the library's entry points

def _library(case, s):
    from diffusion_transformer_qk_gb300 import qknr as Q

    op = case["op"]
    if op.startswith("layer_norm"):
        per = case["seq"] if case["modulated"] else None
        if op == "layer_norm":
            return Q.layer_norm(s["x"], s["weight"], s["bias"], rows_per_batch=per, unit_offset=case["modulated"], eps=EPS)
        return Q.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], rows_per_batch=per,
                                     unit_offset=case["modulated"])
    if op == "qk_norm_rope_backward":
        return Q.qk_norm_rope_packed_backward(s["dout"], s["qkv"], case["heads_q"], case["heads_k"], case["heads_k"],
                                              case["head_dim"], s["gamma_q"], s["gamma_k"], s["cos"], s["sin"],
                                              rope_style=case["style"], eps=EPS, out=torch.empty_like(s["dout"]))
    kw = dict(batch=case["batch"], causal=case["causal"], k_lens=s["k_lens"])
    heads = (case["heads_q"], case["heads_k"], case["head_dim"])
    if op == "attention":
        return Q.attention(s["q"], s["k"], s["v"], *heads, **kw)
    return Q.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], *heads, **kw)


def run(state):
    return list((_library if own else _plain)(state["case"], state))


# ---------------------------------------------------------------------------
# what a pass cannot do without

def _pairs(case):
    """Query-key pairs of one head that some query sees, over the batch."""
    total, n = 0, case["seq_q"]
    for keys in _lengths(case):
        if not case["causal"]:
            total += n * keys
        else:
            # query i sees keys 0 .. i + keys - n
            first = max(0, n - keys)
            a, b = first + keys - n + 1, keys
            total += (a + b) * (n - first) // 2 if n > first else 0
    return total


def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        n = case["batch"] * case["seq"] * case["hidden"]
        sets = (case["batch"] if case["modulated"] else 1) * case["hidden"]
        size, stats = (4 if case["param"] == "fp32" else 2), 8 * case["batch"] * case["seq"]
        if op == "layer_norm":
            return {"bytes": 4 * n + 2 * sets * size + stats, "flops": 8 * n}
        return {"bytes": 6 * n + sets * size + 8 * sets + stats, "flops": 14 * n}
    if op == "qk_norm_rope_backward":
        rows, d = case["batch"] * case["seq"], case["head_dim"]
        n, nv = rows * (case["heads_q"] + case["heads_k"]) * d, rows * case["heads_k"] * d
        return {"bytes": 6 * n + 4 * nv + 2 * case["seq"] * d * (4 if case["table"] == "fp32" else 2) + 16 * d,
                "flops": 16 * n}
    batch, nq, nk, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "heads_q", "heads_k", "head_dim"))
    nq, nk = batch * nq * hq, sum(_lengths(case)) * hk
    if op == "attention":
        return {"bytes": 2 * d * (2 * nq + 2 * nk) + 4 * nq, "flops": 4 * d * hq * _pairs(case)}
    # q, o, do read and dq written; k, v read, dk and dv written whole
    return {"bytes": 2 * d * (4 * nq + 2 * nk + 2 * batch * case["seq_k"] * hk) + 4 * nq,
            "flops": 10 * d * hq * _pairs(case)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_layer_norm(case, s):
    sets = case["batch"] if case["modulated"] else 1
    rows = s["x"].shape[0] // sets
    out = []
    for b in range(sets):
        x = s["x"][b * rows:(b + 1) * rows].double()
        w = s["weight"][b].double() + (1.0 if case["modulated"] else 0.0)
        if case["op"] == "layer_norm":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
            out.append([(x - mean[:, None]) * rstd[:, None] * w + s["bias"][b].double(), mean, rstd])
        else:
            dy, rstd = s["dy"][b * rows:(b + 1) * rows].double(), s["rstd"][b * rows:(b + 1) * rows].double()[:, None]
            xhat = (x - s["mean"][b * rows:(b + 1) * rows].double()[:, None]) * rstd
            g = dy * w
            hidden = x.shape[1]
            a, c = g.sum(1, keepdim=True) / hidden, torch.einsum("rc,rc->r", g, xhat)[:, None] / hidden
            out.append([(g - a - xhat * c) * rstd, torch.einsum("rc,rc->c", dy, xhat)[None], dy.sum(0)[None]])
    return [torch.cat(parts) for parts in zip(*out)]


def _exact_qk_backward(case, s):
    d, hq, hk, seq = case["head_dim"], case["heads_q"], case["heads_k"], case["seq"]
    # the two members of each pair
    if case["style"] == "rotate_half":
        first, second = torch.arange(d // 2, device="cuda"), torch.arange(d // 2, d, device="cuda")
    else:
        first, second = torch.arange(0, d, 2, device="cuda"), torch.arange(1, d, 2, device="cuda")
    cos, sin = s["cos"].double(), s["sin"].double()
    dx, dgamma = s["dout"].double(), [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(2)]
    for h in range(hq + hk):
        gamma, acc = (s["gamma_q"], dgamma[0]) if h < hq else (s["gamma_k"], dgamma[1])
        x, do = s["qkv"][:, h * d:(h + 1) * d].double(), s["dout"][:, h * d:(h + 1) * d].double()
        x, do = x.view(-1, seq, d), do.view(-1, seq, d)
        # o1 = y1 cos1 - y2 sin1, o2 = y2 cos2 + y1 sin2
        dy = torch.empty_like(x)
        dy[..., first] = do[..., first] * cos[:, first] + do[..., second] * sin[:, second]
        dy[..., second] = do[..., second] * cos[:, second] - do[..., first] * sin[:, first]
        ms = x.pow(2).sum(-1, keepdim=True) / d + EPS
        xhat = x / ms.sqrt()
        acc += torch.einsum("bsd,bsd->d", dy, xhat)
        g = dy * gamma.double()
        dx[:, h * d:(h + 1) * d] = ((g - xhat * (g * xhat).sum(-1, keepdim=True) / d) / ms.sqrt()).view(-1, d)
    return [dx, dgamma[0], dgamma[1]]


def _exact_attention(case, s):
    batch, nq, nk, hq, hk, d = (case[k] for k in ("batch", "seq_q", "seq_k", "heads_q", "heads_k", "head_dim"))
    group, scale, back = hq // hk, 1.0 / math.sqrt(d), case["op"] == "attention_backward"
    zeros = lambda rows, heads: torch.zeros(batch * rows, heads * d, dtype=torch.float64, device="cuda")  # noqa: E731
    o, lse = zeros(nq, hq), torch.full((batch, hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = zeros(nq, hq), zeros(nk, hk), zeros(nk, hk)
    for b, keys in enumerate(_lengths(case)):
        # queries from `first` on see a key; query i sees keys 0 .. i + keys - nq where causal
        first = max(0, nq - keys) if case["causal"] else 0
        if keys == 0 or first >= nq:
            continue
        rows, cols = slice(b * nq + first, (b + 1) * nq), slice(b * nk, b * nk + keys)
        hidden = torch.ones(nq - first, keys, dtype=torch.bool, device="cuda").triu(first + keys - nq + 1) if case["causal"] else None
        for h in range(hq):
            hc, kc = slice(h * d, (h + 1) * d), slice(h // group * d, (h // group + 1) * d)
            q, k, v = s["q"][rows, hc].double(), s["k"][cols, kc].double(), s["v"][cols, kc].double()
            t = (q * scale) @ k.T
            if hidden is not None:
                t[hidden] = -math.inf
            if not back:
                lse[b, h, first:] = torch.logsumexp(t, 1)
                o[rows, hc] = torch.softmax(t, 1) @ v
                continue
            p = torch.exp(t - s["lse"][b, h, first:].double()[:, None])
            do = s["do"][rows, hc].double()
            dv[cols, kc] += p.T @ do
            ds = p * (do @ v.T - torch.einsum("rd,rd->r", do, s["o"][rows, hc].double())[:, None])
            dq[rows, hc] = ds @ (k * scale)
            dk[cols, kc] += ds.T @ (q * scale)
    return [dq, dk, dv] if back else [o, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("layer_norm"):
        return _exact_layer_norm(case, s)
    if case["op"] == "qk_norm_rope_backward":
        return _exact_qk_backward(case, s)
    return _exact_attention(case, s)
