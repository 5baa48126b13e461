"""How the tiles of a line are shared out among the CTAs (csrc/attn_plan.cuh and
the spans of csrc/attn_kernel.cuh, restated here; csrc/attn_share.cuh, compiled
from the source): every tile is done exactly once, and the parts that a join
reads are the ones that were written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "diffusion_transformer_qk_gb300", "csrc")
CTAS = 152

# (over, whole, least) of the kinds of tiles: a few queries with some and with all warps of a CTA on a tile; the
# others at head_dim 128 and 64.  A cut costs half of `whole`.
FEW, FEW_ALL, WIDE, NARROW = (4, 12, 4), (4, 5, 4), (2, 12, 6), (3, 24, 6)


@pytest.fixture(scope="module")
def share_cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("share")
    src, so = d / "share.cpp", d / "share.so"
    src.write_text(f'#define __host__\n#define __device__\n#define __forceinline__ inline\n#include "{CSRC}/attn_share.cuh"\n'
                   'extern "C" int share_cut(int o, int u, int over) { return qknr::share_cut(o, u, over); }\n')
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    fn = ctypes.CDLL(str(so)).share_cut
    fn.argtypes, fn.restype = [ctypes.c_int] * 3, ctypes.c_int
    known = {}

    def cut(o, u, over):
        if (o, u, over) not in known:
            known[o, u, over] = fn(o, u, over)
        return known[o, u, over]

    return cut


def blocks(n):
    return -(-n // 128)


def place(cut, tile, o, u, over):
    o = cut(o, u, over)
    return (tile + 1, 0) if o == u else (tile, o)


def plan(cut, costs, heads, kind, near=True, runs=None):
    """(units of the line's items, spans, waves) of attn_plan_kernel."""
    over, most, least = kind
    costs = np.asarray(costs, dtype=np.int64)
    n, line = len(costs), costs
    if near:
        line = costs[sorted(range(n), key=lambda i: (-costs[i], i))]
        runs = [(int((costs > c).sum()), int((costs == c).sum())) for c in line]
    before = np.concatenate([[0], np.cumsum(line)])
    work, tiles = int(before[-1]) * heads, n * heads
    active = min(max(work // least, 1), CTAS)
    each, rest = divmod(work, active)
    share = np.array([each + rest * (c + 1) // active - rest * c // active if c < active else 0 for c in range(CTAS)])
    last, mine = -(-tiles // CTAS), np.zeros(CTAS, dtype=np.int64)
    whole = (int(line.max()) if n else 0) <= most
    waves = last if whole else 0
    if not whole and active == CTAS:
        total, before_last, even, s = np.zeros(CTAS, dtype=np.int64), mine, True, 0
        while s < last:
            for c in range(CTAS):
                t = s * CTAS + (CTAS - 1 - c if s & 1 else c)
                if t < tiles:
                    total[c] += line[t // heads]
            if (total > share + most // 2).any():
                break
            even = even and not (total > share).any() and (s + 1) * CTAS <= tiles
            if even:
                before_last, mine, waves = mine, total.copy(), s + 1
            s += 1
        whole = s == last
        if whole:
            waves = last
        t0 = waves * CTAS
        if not whole and waves > 0 and t0 < tiles and 3 * int((share - mine).sum()) < int(line[t0 // heads]) * CTAS:
            mine, waves = before_last, waves - 1
    spans, upto = [], 0
    for c in range(CTAS + 1):
        at, t0 = (tiles, 0), waves * CTAS
        if c < active and not whole and t0 < tiles:
            first = runs[t0 // heads][0]
            x = int(before[first]) * heads + (t0 - first * heads) * int(line[t0 // heads]) + upto
            if x < work:
                i = int(np.searchsorted(before[:n] * heads, x, side="right")) - 1
                first, u = runs[i][0], int(line[i])
                off = x - int(before[first]) * heads
                at = place(cut, first * heads + off // u, off % u, u, over)
        if c < active:
            upto += int(share[c] - mine[c])
        spans.append(at)
    return line, spans, waves


def check(line, heads, spans, waves):
    """The pieces as attn_piece takes them, the parts as the joins read them."""
    assert all(a <= b for a, b in zip(spans, spans[1:])), "shares out of order"
    tiles, parts, whole = len(line) * heads, {}, {}
    for c in range(CTAS):
        for s in range(waves):
            t = s * CTAS + (CTAS - 1 - c if s & 1 else c)
            if t < tiles:
                whole[t] = whole.get(t, 0) + 1
        (t, u0), to = spans[c], spans[c + 1]
        while t < to[0] or (t == to[0] and to[1] > 0):
            u = int(line[t // heads])
            u1 = to[1] if t == to[0] else u
            slot = 2 * c if u0 > 0 else 2 * c + 1 if u1 < u else -1
            assert u0 <= u1
            if slot < 0:
                whole[t] = whole.get(t, 0) + 1
            else:
                assert slot not in parts
                parts[slot] = (t, u0, u1)
            t, u0 = t + 1, 0
    cut = set()
    for c in range(1, CTAS):
        t, u = spans[c]
        if u == 0 or (spans[c - 1][0] == t and spans[c - 1][1] > 0):
            continue
        assert t not in cut
        cut.add(t)
        began = sum(x[0] < t or x == (t, 0) for x in spans) - 1
        at = 0
        for i in range(1 + sum(x[0] == t and x[1] > 0 for x in spans)):
            slot = 2 * began + 1 if i == 0 else 2 * (began + i)
            assert slot in parts and parts[slot][:2] == (t, at), f"tile {t}: slot {slot} holds {parts.get(slot)}, not a part from {at} on"
            at = parts.pop(slot)[2]
        assert at == int(line[t // heads])
    assert not parts, "parts that no join reads"
    assert all(whole.get(t, 0) == (t not in cut) for t in range(tiles))


@pytest.mark.parametrize("over", [2, 3, 4])
def test_a_later_boundary_stays_later(share_cut, over):
    for u in range(over, 400):
        at = [share_cut(o, u, over) for o in range(u)]
        assert at == sorted(at) and at[0] == 0 and at[-1] in (0, u)
        # in a tile: behind two blocks, before two blocks and the tile's end
        assert all(x in (0, u) or 2 <= x <= u - over - 2 for x in at)
        # where a tile may be cut, it is cut where it was asked for
        assert all(at[o] == o for o in range(2, u - over - 1))


def few(lens):
    return [blocks(n) + 4 for n in lens]


def queries(lens, rows, over):
    return [blocks(n) + over for n in lens for _ in range(-(-n // rows))]


@pytest.mark.parametrize("costs,heads,kind", [
    (few([1000] * 39 + [640] * 63), 2, FEW_ALL),                     # a query each
    (few([1152] + [640] * 63), 4, FEW_ALL),                          # own keys beside a prefix
    (queries([3000] * 3 + [512] * 33, 256, 3), 3, NARROW),           # forward
    (queries([3375] * 2 + [512] * 28, 128, 3), 2, NARROW),           # dk and dv
    ([], 3, WIDE), ([6], 1, FEW_ALL), ([2000], 1, WIDE), ([7] * 200, 1, FEW_ALL),
])
def test_each_tile_is_done_once(share_cut, costs, heads, kind):
    check(*(lambda p: (p[0], heads, *p[1:]))(plan(share_cut, costs, heads, kind)))


@pytest.mark.parametrize("kind", [FEW, FEW_ALL, WIDE, NARROW])
@pytest.mark.parametrize("near", [True, False])
def test_each_tile_is_done_once_at_random(share_cut, kind, near):
    for seed in range(250):
        gen = np.random.Generator(np.random.PCG64(seed))
        n, most, heads = int(gen.integers(1, 250)), int(gen.integers(1, 60)), int(gen.integers(1, 9))
        if seed % 2:
            units = gen.integers(0, most + 1, size=n)
        else:                                     # long ones and short ones
            units = np.where(gen.random(n) < gen.random(), most, gen.integers(1, 8))
        costs = (units + kind[0]).tolist()
        runs = None
        if not near:                              # the sequences' order, each sequence's items a run
            runs, k = [], 0
            while k < n:
                m = min(int(gen.integers(1, 9)), n - k)
                costs[k:k + m] = [costs[k]] * m
                runs += [(k, m)] * m
                k += m
        line, spans, waves = plan(share_cut, costs, heads, kind, near, runs)
        check(line, heads, spans, waves)


def even_spans(cut, line, heads, over, least):
    """table_span and uniform_span: equal stretches of the line, head by head."""
    before = np.concatenate([[0], np.cumsum(line)])
    units, n = int(before[-1]), len(line)
    work = units * heads
    active = min(max(work // least, 1), CTAS)
    spans = []
    for c in range(CTAS + 1):
        x = work // active * c + work % active * c // active if c < active else work
        if x >= work:
            spans.append((n * heads, 0))
            continue
        h, off = divmod(x, units)
        i = int(np.searchsorted(before[:n], off, side="right")) - 1
        spans.append(place(cut, h * n + i, off - int(before[i]), int(line[i]), over))
    return spans


@pytest.mark.parametrize("kind", [FEW_ALL, WIDE, NARROW])
@pytest.mark.parametrize("uniform", [True, False])
def test_equal_stretches_do_each_tile_once(share_cut, kind, uniform):
    for seed in range(300):
        gen = np.random.Generator(np.random.PCG64(seed))
        n, most, heads = int(gen.integers(1, 33)), int(gen.integers(1, 300 if seed % 3 else 12)), int(gen.integers(1, 25))
        units = gen.integers(0, most + 1, size=n)
        line = np.full(n, int(units[0])) if uniform else units
        line = line + kind[0]
        spans = even_spans(share_cut, line, heads, kind[0], kind[2])
        check(np.tile(line, heads), 1, spans, 0)
