"""Attention over packed sequences and its backward pass against the fp64
oracle, sequence by sequence and with the bounds of attention itself."""
import numpy as np
import pytest
import torch

import tests.test_attention_gpu as TA
from diffusion_transformer_qk_gb300 import qknr as Q
from oracle import sequence_oracle as S
from tests.gpu_util import TORCH
from tests.training_util import f64, normal, same_bits

pytestmark = pytest.mark.gpu

KEPT = 7.0                            # what rows of no sequence hold before a call


@pytest.fixture(scope="module", autouse=True)
def _lib(built_lib, cuda_device):
    Q.load()
    Q.status_buffer().zero_()
    yield
    assert Q.read_status() == 0, "a kernel reported a wait timeout"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(lens, first=0):
    return [first, *(first + np.cumsum(lens)).tolist()]


def make(lens_q, lens_k, Hq, Hk, D, dtype="bf16", causal=False, seed=0, before=0, behind=0, scale=None, size=1.0,
         garbage=True):
    """lens_k None: one packed qkv buffer, self-attention."""
    gen, td = np.random.Generator(np.random.PCG64(seed)), TORCH[dtype]
    sq = starts(lens_q, before)
    rows_q = sq[-1] + behind
    if lens_k is None:
        sk, rows_k = sq, rows_q
        buf = normal(gen, (rows_q, (Hq + 2 * Hk) * D), td, size)
        q, k, v = buf[:, :Hq * D], buf[:, Hq * D:(Hq + Hk) * D], buf[:, (Hq + Hk) * D:]
    else:
        sk = starts(lens_k, 2 * before)
        rows_k = sk[-1] + behind // 2
        q, k, v = (normal(gen, (n, H * D), td, size) for n, H in ((rows_q, Hq), (rows_k, Hk), (rows_k, Hk)))
    do = normal(gen, (rows_q, Hq * D), td, 0.3)
    if garbage:
        for t, s, x in ((q, sq, "nan"), (do, sq, "nan"), (k, sk, "nan"), (v, sk, "inf")):
            t[:s[0]] = float(x)
            t[s[-1]:] = float(x)
    return dict(q=q, k=k, v=v, do=do, sq=sq, sk=sk, Hq=Hq, Hk=Hk, D=D, dtype=dtype, causal=causal,
                scale=1 / np.sqrt(D) if scale is None else float(np.float32(scale)), one=lens_k is None)


def call(s, **kw):
    return Q.attention_packed(s["q"], s["k"], s["v"], s["Hq"], s["Hk"], s["D"], ints(s["sq"]),
                              None if s["one"] else ints(s["sk"]), scale=s["scale"], causal=s["causal"], **kw)


def call_backward(s, do, o, lse, **kw):
    return Q.attention_packed_backward(do, s["q"], s["k"], s["v"], o, lse, s["Hq"], s["Hk"], s["D"], ints(s["sq"]),
                                       None if s["one"] else ints(s["sk"]), scale=s["scale"], causal=s["causal"], **kw)


def each(s):
    """The sequences as samples of their own: (its dict, query rows, key rows)."""
    for (a, b), (c, d) in S.sequences(s["sq"], s["sk"], s["q"].shape[0], s["k"].shape[0]):
        one = dict(q=s["q"][a:b], k=s["k"][c:d], v=s["v"][c:d], B=1, Hq=s["Hq"], Hk=s["Hk"], D=s["D"], scale=s["scale"],
                   causal=s["causal"], q_lens=None, k_lens=None)
        yield one, slice(a, b), slice(c, d)


def outside(n, used):
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    for r in used:
        keep[r] = False
    return keep


def check_forward(s, o, lse):
    used = []
    for one, rows, keys in each(s):
        used.append(rows)
        if rows.stop == rows.start:
            continue
        if keys.stop == keys.start:
            assert not o[rows].float().any() and torch.isneginf(lse[:, rows]).all()
            continue
        TA.check_forward(one, s["dtype"], o[rows], lse[:, rows])
    keep = outside(o.shape[0], used)
    assert (o[keep] == KEPT).all() and (lse[:, keep] == KEPT).all()


def check_backward(s, o, lse, dq, dk, dv):
    used_q, used_k = [], []
    for one, rows, keys in each(s):
        used_q.append(rows)
        used_k.append(keys)
        if rows.stop == rows.start or keys.stop == keys.start:
            assert not any(t.float().any() for t in (dq[rows], dk[keys], dv[keys]))
            continue
        TA.check_backward(one, s["dtype"], s["do"][rows], o[rows], lse[:, rows], dq[rows], dk[keys], dv[keys])
    assert (dq[outside(dq.shape[0], used_q)] == KEPT).all()
    keep = outside(dk.shape[0], used_k)
    assert (dk[keep] == KEPT).all() and (dv[keep] == KEPT).all()


def kept(*shape, dtype=torch.float32):
    return torch.full(shape, KEPT, dtype=dtype, device="cuda")


def forward(s):
    td = TORCH[s["dtype"]]
    o, lse = kept(*s["q"].shape, dtype=td), kept(s["Hq"], s["q"].shape[0])
    got = call(s, out=o, lse=lse)
    assert got[0] is o and got[1] is lse
    check_forward(s, o, lse)
    return o, lse


def both(*args, **kw):
    s = make(*args, **kw)
    td = TORCH[s["dtype"]]
    o, lse = forward(s)
    grads = [kept(*t.shape, dtype=td) for t in (s["q"], s["k"], s["v"])]
    call_backward(s, s["do"], o, lse, dq=grads[0], dk=grads[1], dv=grads[2])
    check_backward(s, o, lse, *grads)
    return s, o, lse, grads


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("fp16", 64), ("fp16", 128)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens", [[1], [17], [128], [300], [129, 127, 256, 1, 0, 64], [40, 1, 31, 500, 260], [0, 0, 33, 0]])
def test_self_attention(lens, causal, dtype, D):
    both(lens, None, 4, 2, D, dtype=dtype, causal=causal, seed=sum(lens))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [([300, 5, 77], [40, 700, 0]), ([64, 0, 200], [64, 100, 33]), ([129], [1]),
                                           ([400, 31], [399, 600]), ([0, 0], [100, 30]), ([50, 60], [0, 0])])
def test_keys_of_other_lengths(lens_q, lens_k, causal, D):
    # with causal, the first queries of sequences with fewer keys see none
    both(lens_q, lens_k, 6, 3, D, causal=causal, seed=len(lens_q) + sum(lens_k))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("before,behind", [(3, 0), (0, 200), (37, 90)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_of_no_sequence_are_left(before, behind, dtype, causal):
    both([130, 60, 333], None, 2, 1, 64, dtype=dtype, causal=causal, before=before, behind=behind, seed=5)
    both([30, 60], [200, 133], 2, 2, 128, dtype=dtype, causal=causal, before=before, behind=behind, seed=6)
    both([1, 3], [200, 133], 2, 2, 128, dtype=dtype, causal=causal, before=before, behind=behind, seed=7)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (8, 8), (12, 3), (16, 1), (40, 2)])
@pytest.mark.parametrize("lens_q,lens_k", [([1, 1, 1], [700, 1, 64]), ([1] * 20, [150] * 20), ([2, 16, 0, 30], [512, 17, 40, 2000]),
                                           ([1], [5000]), ([1, 1, 1], [0, 3, 0])])
def test_a_few_queries(lens_q, lens_k, Hq, Hk, causal, D):
    forward(make(lens_q, lens_k, Hq, Hk, D, causal=causal, seed=Hq + sum(lens_k), dtype="fp16" if Hq == 8 else "bf16"))


def test_many_short_sequences():
    # more sequences than the planning CTA has threads
    gen = np.random.Generator(np.random.PCG64(8))
    lens = gen.integers(0, 40, size=2500).tolist()
    s = make(lens, None, 2, 1, 64, causal=True, seed=9)
    o, lse = kept(*s["q"].shape, dtype=torch.bfloat16), kept(2, s["q"].shape[0])
    call(s, out=o, lse=lse)
    td = [kept(*t.shape, dtype=torch.bfloat16) for t in (s["q"], s["k"], s["v"])]
    call_backward(s, s["do"], o, lse, dq=td[0], dk=td[1], dv=td[2])
    H = lambda t, h: f64(t).reshape(-1, h, 64)  # noqa: E731
    ref, rl = S.packed(H(s["q"], 2), H(s["k"], 1), H(s["v"], 1), s["scale"], True, s["sq"], s["sk"])
    assert np.abs(H(o, 2) - ref).max() < 3e-2 and np.abs(f64(lse) - rl).max() < 1e-4
    refs = S.packed_backward(H(s["do"], 2), H(s["q"], 2), H(s["k"], 1), H(s["v"], 1), H(o, 2), f64(lse), s["scale"], True, s["sq"],
                             s["sk"])
    for got, r, h in zip(td, refs, (2, 1, 1)):
        assert np.abs(H(got, h) - r).max() < 3e-2


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_long_and_short_together(D, causal):
    # one long sequence whose tiles are cut among the CTAs, and short ones
    both([2500, 3, 700, 129], None, 2, 1, D, causal=causal, seed=10)


@pytest.mark.parametrize("causal", [False, True])
def test_few_tiles_over_many_keys(causal):
    both([256], [9000], 1, 1, 128, causal=causal, seed=11)
    both([20, 17], [4000, 6000], 3, 1, 64, causal=causal, seed=12, dtype="fp16")


@pytest.mark.parametrize("bad", [[0, 300, 100, 450], [-5, 300, 450, 10 ** 9], [2 ** 31 - 1, 0, 5, 0], [450, 0, 450, 0],
                                 [-2 ** 31, -1, 0, 450], [100, 100, 100, 100]])
def test_starts_out_of_order_or_range(bad):
    # clamped: no row is in two sequences, nothing outside the tensors
    s = make([100, 200, 150], None, 2, 1, 64, causal=True, seed=13)
    s["sq"] = s["sk"] = bad
    o, lse = kept(*s["q"].shape, dtype=torch.bfloat16), kept(2, 450)
    call(s, out=o, lse=lse)
    check_forward(s, o, lse)
    grads = [kept(*t.shape, dtype=torch.bfloat16) for t in (s["q"], s["k"], s["v"])]
    call_backward(s, s["do"], o, lse, dq=grads[0], dk=grads[1], dv=grads[2])
    check_backward(s, o, lse, *grads)
    # a few queries
    s["sq"], s["one"] = [0, 1, 1, 5], False
    o.fill_(KEPT)
    lse.fill_(KEPT)
    Q.attention_packed(s["q"][:8], s["k"], s["v"], 2, 1, 64, ints(s["sq"]), ints(bad), scale=s["scale"], causal=True, out=o[:8],
                       lse=lse.view(-1)[:16].view(2, 8))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_sequence_of_nans_stays_alone(dtype):
    s = make([200, 90, 310], None, 4, 2, 64, dtype=dtype, causal=True, seed=14)
    o, lse = call(s)
    grads = call_backward(s, s["do"], o, lse)
    bad = slice(200, 290)
    for t, x in ((s["q"], "nan"), (s["k"], "inf"), (s["v"], "nan")):
        t[bad] = float(x)
    o2, lse2 = call(s)
    keep = outside(600, [bad])
    assert same_bits(o2[keep], o[keep]) and same_bits(lse2[:, keep], lse[:, keep])
    do = s["do"].clone()
    do[bad] = float("nan")
    grads2 = call_backward(s, do, o2, lse2)
    for a, b in zip(grads2, grads):
        assert torch.isfinite(a[keep].float()).all()
        if dtype == "bf16":
            assert same_bits(a[keep], b[keep])


def test_same_as_attention_of_equal_lengths():
    # three sequences of 300 are a batch of three
    s = make([300] * 3, None, 4, 2, 128, dtype="fp16", causal=True, seed=15)
    o, lse = call(s)
    o1, lse1 = Q.attention(s["q"], s["k"], s["v"], 4, 2, 128, batch=3, causal=True, scale=s["scale"])
    assert (o.float() - o1.float()).abs().max() < 2e-3
    assert (lse.view(4, 3, 300).transpose(0, 1) - lse1).abs().max() < 1e-5


def test_equal_calls_give_equal_bits_graph_and_streams():
    s = make([700, 30, 1200, 5], None, 8, 2, 64, causal=True, seed=16)
    o, lse = call(s)
    grads = call_backward(s, s["do"], o, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o2, lse2 = call(s, stream=side)
        with torch.cuda.stream(side):
            again = call_backward(s, s["do"], o2, lse2)
        side.synchronize()
        assert same_bits(o, o2) and same_bits(lse, lse2) and all(same_bits(a, b) for a, b in zip(again, grads))
    # a captured call reads the starts that are there when it is replayed
    sq, graph = ints(s["sq"]), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    args = (s["Hq"], s["Hk"], s["D"], sq)
    with torch.cuda.graph(graph):
        go, gl = Q.attention_packed(s["q"], s["k"], s["v"], *args, scale=s["scale"], causal=True)
        gg = Q.attention_packed_backward(s["do"], s["q"], s["k"], s["v"], go, gl, *args, scale=s["scale"], causal=True)
    for lens in ([700, 30, 1200, 5], [5, 900, 930, 100], [1935, 0, 0, 0], [484, 484, 484, 483]):
        sq.copy_(ints(starts(lens)))
        graph.replay()
        e = Q.attention_packed(s["q"], s["k"], s["v"], *args, scale=s["scale"], causal=True)
        f = Q.attention_packed_backward(s["do"], s["q"], s["k"], s["v"], *e, *args, scale=s["scale"], causal=True)
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip((go, gl, *gg), (*e, *f)))


def test_gradients_into_one_buffer_and_two_calls_of_one_workspace():
    s = make([129, 400, 64], None, 2, 2, 64, seed=17)
    o, lse = call(s)
    plain = call_backward(s, s["do"], o, lse)
    d = torch.empty_like(s["q"]._base if s["q"]._base is not None else s["q"])
    cols = d.split(128, dim=1)
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o2, _ = call(s, workspace=ws)
        call_backward(s, s["do"], o2, lse, dq=cols[0], dk=cols[1], dv=cols[2], workspace=ws)
        assert same_bits(o, o2)
    assert all(same_bits(a, b) for a, b in zip(cols, plain))


def test_waits_are_bounded():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(flags=Q.FLAG_TEST_STALL, wait_limit_ns=20_000_000, dev_status=word)
    s = make([300, 40], None, 2, 1, 64, seed=18)
    o, lse = call(s)
    few = make([1, 1], [300, 200], 2, 1, 64, seed=19)
    for f in (lambda: call(s, **kw), lambda: call(few, **kw), lambda: call_backward(s, s["do"], o, lse, **kw)):
        word.zero_()
        f()
        assert int(word.item()) == Q.ERR_TIMEOUT
    both([300, 40], None, 2, 1, 64, seed=18)


@pytest.mark.parametrize("lens,Hq,Hk,D", [([2800, 591, 619], 12, 12, 128), ([686, 560, 1844], 8, 8, 128), ([3000, 200, 90], 6, 2, 64)])
@pytest.mark.parametrize("few", [False, True])
def test_a_workspace_full_of_nan(lens, Hq, Hk, D, few):
    # whatever a workspace held, every part that a join adds up has been written: also those of CTAs whose share of the
    # work left over is nothing, which the first two shapes have inside a tile
    s = make([3] * len(lens) if few else lens, lens if few else None, Hq, Hk, D, seed=20)
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")
    o, lse = call(s, workspace=ws)
    o2, lse2 = call(s)
    assert same_bits(o, o2) and same_bits(lse, lse2)
    ws.fill_(255)
    grads = call_backward(s, s["do"], o, lse, workspace=ws)
    assert all(same_bits(a, b) for a, b in zip(grads, call_backward(s, s["do"], o, lse)))
    one, rows, keys = list(each(s))[1]
    TA.check_forward(one, s["dtype"], o[rows], lse[:, rows])
    TA.check_backward(one, s["dtype"], s["do"][rows], o[rows], lse[:, rows], grads[0][rows], grads[1][keys], grads[2][keys])


def test_lengths_at_random():
    # the plan's every turn: some sequences or many, tiles that go out whole and tiles that are cut
    for seed in range(24):
        gen = np.random.Generator(np.random.PCG64(100 + seed))
        B = int(gen.integers(1, 40 if seed % 2 else 6))
        most = int(gen.integers(1, 200 if B > 6 else 2500))
        lens = gen.integers(0, most + 1, size=B).tolist()
        Hk, group, D = int(gen.integers(1, 5)), int(gen.choice([1, 2, 3])), int(gen.choice([64, 128]))
        lens_k = None if seed % 3 else gen.integers(0, most + 1, size=B).tolist()
        s = make(lens, lens_k, Hk * group, Hk, D, causal=bool(seed & 4), dtype="fp16" if seed & 8 else "bf16", seed=seed)
        o, lse = call(s)
        grads = call_backward(s, s["do"], o, lse)
        kw = dict(causal=s["causal"], scale=s["scale"])
        for one, rows, keys in each(s):
            a, b = rows.stop - rows.start, keys.stop - keys.start
            if a == 0 or b == 0:
                continue
            # the same sequence through attention() as a sample of its own: a rounding of o or of a gradient apart, and
            # p's and ds's own roundings (h each of the terms' sum, which random signs keep below 1 here)
            o1, l1 = Q.attention(one["q"], one["k"], one["v"], s["Hq"], s["Hk"], D, **kw)
            tol = 4 * 2.0 ** (-11 if s["dtype"] == "fp16" else -8)
            fin = torch.isfinite(l1[0])
            assert torch.equal(fin, torch.isfinite(lse[:, rows])) and (l1[0] - lse[:, rows])[fin].abs().max() < 1e-4
            assert (o1.float() - o[rows].float()).abs().max() <= tol * max(1.0, float(o1.float().abs().max()))
            ref = Q.attention_backward(s["do"][rows], one["q"], one["k"], one["v"], o[rows], lse[:, rows].contiguous()[None],
                                       s["Hq"], s["Hk"], D, **kw)
            for x, y in zip((grads[0][rows], grads[1][keys], grads[2][keys]), ref):
                assert (x.float() - y.float()).abs().max() <= tol * max(1.0, float(y.float().abs().max())), (seed, a, b)


@pytest.mark.parametrize("lens_q,lens_k", [([1, 1], [0, 0]), ([3, 0, 9], [0, 0, 0]), ([0, 0], [0, 0]), ([1] * 40, [0] * 39 + [3])])
@pytest.mark.parametrize("causal", [False, True])
def test_a_few_queries_without_keys(lens_q, lens_k, causal):
    both(lens_q, lens_k, 4, 2, 64, causal=causal, seed=21, behind=4)


def test_more_items_than_the_plan_sorts():
    # 1100 tiles of a head and 300 sequences: the plan keeps the sequences' order.  Checked against attention() where
    # lengths repeat, so that one batch of it does them all
    lens = [40, 700, 900] * 100
    s = make(lens, None, 2, 1, 64, causal=True, seed=22)
    o, lse = call(s)
    grads = call_backward(s, s["do"], o, lse)
    for n in set(lens):
        at = [a for a, m in zip(s["sq"], lens) if m == n]
        pick = torch.cat([torch.arange(a, a + n, device="cuda") for a in at])
        q, k, v, do = (s[x][pick].contiguous() for x in ("q", "k", "v", "do"))
        kw = dict(batch=len(at), causal=True, scale=s["scale"])
        o1, l1 = Q.attention(q, k, v, 2, 1, 64, **kw)
        mine = lse[:, pick].view(2, len(at), n).transpose(0, 1).contiguous()
        # a rounding of o apart, and p's own roundings
        assert (o1.float() - o[pick].float()).abs().max() <= 4 * 2.0 ** -8 * float(o1.float().abs().max())
        assert (l1 - mine).abs().max() < 1e-4
        ref = Q.attention_backward(do, q, k, v, o[pick].contiguous(), mine, 2, 1, 64, **kw)
        for a, b in zip(grads, ref):
            assert (a[pick].float() - b.float()).abs().max() <= 4 * 2.0 ** -8 * max(1.0, float(b.float().abs().max()))


def test_outputs_beside_inputs():
    s = make([129, 64, 300], None, 2, 1, 64, causal=True, seed=24)
    o, lse = call(s)
    wide = torch.full((493, 2 * 128 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :128] = s["q"]
    o2, lse2 = call(dict(s, q=wide[:, :128]), out=wide[:, 128:256])
    assert same_bits(o, o2) and same_bits(lse, lse2)
    assert same_bits(wide[:, :128], s["q"]) and (wide[:, 256:] == 7.0).all()


def test_two_streams_at_once():
    # two calls in flight, each with its own workspace from the binding
    a, b = make([900, 30, 2000], None, 4, 2, 64, causal=True, seed=25), make([1] * 20, [700] * 20, 8, 2, 128, seed=26)
    ref = [call(s) for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert same_bits(o, ref[i][0]) and same_bits(lse, ref[i][1])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens_q,lens_k", [([2, 1, 2, 4], [1, 1, 1, 1]), ([300, 130, 1], [1, 2, 300]), ([200, 1, 70, 129], None),
                                           ([129, 400], [65, 300])])
def test_a_single_key_has_no_gradient_of_its_score(lens_q, lens_k, causal, dtype, D):
    # its probability is 1 whatever the score: exact zeros, not what dp - delta leaves of rounding
    s, o, lse, (dq, dk, dv) = both(lens_q, lens_k, 4, 2, D, dtype=dtype, causal=causal, seed=31)
    alone = 0
    for (a, b), (c, d) in S.sequences(s["sq"], s["sk"], s["q"].shape[0], s["k"].shape[0]):
        if d - c == 1:
            assert not dq[a:b].float().any() and not dk[c:d].float().any()
            alone += 1
        elif causal and 0 <= (b - a) - (d - c) < b - a:
            # the first query that sees a key sees one
            assert not dq[b - (d - c)].float().any()
            alone += 1
    assert alone or lens_k == [65, 300] and not causal
    # and the others' gradients are there
    assert dv.float().any()


@pytest.mark.parametrize("D", [64, 128])
def test_calls_on_one_workspace_in_a_row(D):
    # passes of one call run beside each other, calls do not: with one workspace for all of them, nothing waited for
    a = make([2800, 591, 619], None, 12, 12, D, dtype="fp16", seed=41, garbage=False)
    b = make([1100, 900, 40, 1500], None, 8, 2, D, dtype="fp16", causal=True, seed=42, garbage=False)
    gen = np.random.Generator(np.random.PCG64(43))
    q, k, v, pk, pv = (normal(gen, (n, H * D), torch.float16, 1.0)
                       for n, H in ((48, 8), (48 * 64, 2), (48 * 64, 2), (3000, 2), (3000, 2)))

    at = [ints(s["sq"]) for s in (a, b)]

    def calls(**kw):
        got = []
        for s, sq in zip((a, b), at):
            args = (s["Hq"], s["Hk"], s["D"], sq)
            kw.update(scale=s["scale"], causal=s["causal"])
            o, lse = Q.attention_packed(s["q"], s["k"], s["v"], *args, **kw)
            got += [o, lse, *Q.attention_packed_backward(s["do"], s["q"], s["k"], s["v"], o, lse, *args, **kw)]
            got += Q.attention_prefix(q, k, v, pk, pv, 8, 2, D, batch=48, **kw)
        return got

    apart = calls()
    torch.cuda.synchronize()
    ws = torch.full((1 << 28,), 255, dtype=torch.uint8, device="cuda")
    rounds = [calls(workspace=ws) for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = calls(workspace=ws)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    for got in (*rounds, captured):
        assert all(same_bits(x, y) for x, y in zip(got, apart))
