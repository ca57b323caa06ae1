"""CPU model of how chunk attention divides its work: the same integer arithmetic
as chunk_attention.cuh (ChunkSeq, ChunkWalk, ChunkLine, the merge's plan), checked
for every key tile of every unit being done exactly once, every partial result
written once and read once, and every cut unit merged exactly once."""
import os
import re

import numpy as np
import pytest

SRC = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_26_gb300",
                        "csrc", "chunk_attention.cuh")).read()


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", SRC).group(1))


KEYS, UNIT_KEYS, LEAST = constant("kChunkKeys"), constant("kUnitKeys"), constant("kLeastKeys")


class Seq:
    def __init__(self, n, ctx, T, whole=False):
        self.n, self.ctx, self.T, self.tt, self.whole = n, ctx, T, 2 * T, whole
        self.units = -(-n // self.tt)
        self.before = max(ctx - n, 0)
        self.line = self.start(self.units - 1) + self.before + n + UNIT_KEYS if n > 0 else 0
        if whole:
            self.line = self.units

    def start(self, i):
        if self.whole:
            return i
        return i * (self.before + UNIT_KEYS) + self.tt * (i * (i + 1) // 2)

    def cost(self, i):
        if self.whole:
            return 1
        return min((i + 1) * self.tt, self.n) + self.before + UNIT_KEYS

    def tiles(self, i):
        tokens, first = min(self.tt, self.n - i * self.tt), self.ctx - self.n + i * self.tt
        a = -(-max(first + min(tokens, self.T), 0) // KEYS)
        b = -(-max(first + tokens, 0) // KEYS) if tokens > self.T else 0
        return a, b


def tile_at(offset, cost, tiles):
    return tiles if offset >= cost else min(offset // KEYS, tiles)


def line_cut(total, parts, c):
    return total // parts * c + total % parts * c // parts


def locate(seqs, heads, x):
    at = 0
    for b, s in enumerate(seqs):
        if x < at + s.line * heads:
            rest = x - at
            f = np.float32
            kvh, steps = min(int(f(rest) / f(s.line)), heads - 1), 0
            while kvh > 0 and kvh * s.line > rest:
                kvh, steps = kvh - 1, steps + 1
            while (kvh + 1) * s.line <= rest:
                kvh, steps = kvh + 1, steps + 1
            assert steps <= 1
            rest -= kvh * s.line
            p, y = f(s.before + UNIT_KEYS) + f(0.5) * f(s.tt), f(rest)
            i = rest if s.whole else int(f(2) * y / (p + np.sqrt(p * p + f(2) * f(s.tt) * y)))
            i = min(max(i, 0), s.units - 1)
            steps = 0
            while i > 0 and s.start(i) > rest:
                i, steps = i - 1, steps + 1
            while i + 1 < s.units and s.start(i + 1) <= rest:
                i, steps = i + 1, steps + 1
            assert steps <= 2
            return b, kvh, i, x - (rest - s.start(i))
        at += s.line * heads
    raise AssertionError("past the end of the line")


def plan(new, ctx, heads, group, grid, whole=False):
    T = 128 // group
    seqs = [Seq(n, c, T, whole) for n, c in zip(new, ctx)]
    total = sum(s.line * heads for s in seqs)
    parts = max(1, min(grid, total if whole else total // LEAST))
    pieces = []                       # (cta, unit, t0, t1, slot)
    for cta in range(parts):
        at, stop = line_cut(total, parts, cta), line_cut(total, parts, cta + 1)
        if at >= stop:
            continue
        b, kvh, i, unit_at = locate(seqs, heads, at)
        while at < stop and b < len(seqs):
            s = seqs[b]
            cost, tiles = s.cost(i), max(s.tiles(i))
            begin, end = at - unit_at, min(stop - unit_at, cost)
            t0, t1 = tile_at(begin, cost, tiles), tile_at(end, cost, tiles)
            slot = -1 if (t0, t1) == (0, tiles) else 2 * cta + 1 if t0 == 0 else 2 * cta
            if t0 < t1 or (tiles == 0 and begin == 0):
                pieces.append((cta, (b, kvh, i), t0, t1, slot))
            at = unit_at + end
            if end == cost:
                unit_at += cost
                i += 1
                if i == s.units:
                    i, kvh = 0, kvh + 1
                    if kvh == heads:
                        kvh, b = 0, b + 1
                        while b < len(seqs) and seqs[b].n == 0:
                            b += 1
    return seqs, total, parts, pieces


def merges(grid, pieces):
    """What every merge CTA reads: (unit, [slots]), from how each CTA's part begins."""
    cuts = [None] * grid
    for cta, unit, t0, t1, slot in reversed(pieces):
        cuts[cta] = (unit, t0 > 0, slot)
    first = {}
    for cta, unit, t0, t1, slot in pieces:
        first.setdefault(cta, (unit, t0, t1))
    opened = {}
    for cta, (unit, t0, t1) in first.items():
        opened[cta] = t0 > 0 and t1 < max(p[3] for p in pieces if p[1] == unit)
    for c in range(1, grid):
        if not cuts[c] or not cuts[c][1] or (cuts[c - 1] and cuts[c - 1][1] and opened[c - 1]):
            continue
        got, x = [2 * c - 1, 2 * c], c
        while opened[x] and x + 1 < grid:
            x += 1
            got.append(2 * x)
        yield cuts[c][0], got


def check(new, ctx, heads, group, grid, whole=False):
    seqs, total, parts, pieces = plan(new, ctx, heads, group, grid, whole)
    done, slots = {}, {}
    for cta, unit, t0, t1, slot in pieces:
        done.setdefault(unit, []).append((t0, t1, slot))
        if slot >= 0:
            assert 0 <= slot < 2 * grid and slot not in slots
            slots[slot] = (unit, t0, t1)
    units = {(b, h, i) for b, s in enumerate(seqs) for h in range(heads) for i in range(s.units)}
    assert set(done) == units
    cut = set()
    for unit, got in done.items():
        tiles = max(seqs[unit[0]].tiles(unit[2]))
        got.sort()
        assert got[0][0] == 0 and got[-1][1] == tiles
        assert all(x[1] == y[0] for x, y in zip(got, got[1:]))
        assert (len(got) == 1) == (got[0][2] == -1)
        if len(got) > 1:
            cut.add(unit)
    merged = list(merges(grid, pieces))
    assert {u for u, _ in merged} == cut and len(merged) == len(cut)
    for unit, got in merged:
        ranges = [slots.pop(s) for s in got]
        assert all(u == unit for u, _, _ in ranges) and ranges[0][1] == 0
        assert all(a[2] == b[1] for a, b in zip(ranges, ranges[1:])) and ranges[-1][2] == max(seqs[unit[0]].tiles(unit[2]))
    assert not slots
    return parts, pieces


@pytest.mark.parametrize("group", range(1, 9))
@pytest.mark.parametrize("grid", [1, 7, 152])
def test_every_tile_once(group, grid):
    rng = np.random.default_rng(group * 1000 + grid)
    for trial in range(25):
        B = int(rng.integers(1, 9))
        kind = trial % 5
        if kind == 0:
            new, before = rng.integers(0, 4, B), rng.integers(0, 300, B)
        elif kind == 1:
            new, before = rng.integers(0, 700, B), np.zeros(B, int)
        elif kind == 2:
            new, before = rng.integers(1, 2, B), rng.integers(0, 40000, B)
        elif kind == 3:
            new, before = rng.integers(0, 300, B), rng.integers(0, 5000, B)
        else:
            new, before = rng.integers(0, 600, B), -rng.integers(0, 900, B)  # contexts shorter than the chunk
        ctx = np.maximum(new + before, 0)
        check(new.tolist(), ctx.tolist(), int(rng.integers(1, 9)), group, grid)


@pytest.mark.parametrize("group", range(1, 9))
@pytest.mark.parametrize("grid", [1, 7, 152])
def test_whole_units_are_never_cut(group, grid):
    """The line of units: no partial results, one unit a CTA where there are enough (more
    units than CTAs only where the offsets are not what they should be)."""
    rng = np.random.default_rng(group + grid)
    for trial in range(20):
        B = int(rng.integers(1, 9))
        new = rng.integers(0, 200, B)
        ctx = np.maximum(new + rng.integers(-100, 800, B), 0)
        heads = int(rng.integers(1, 9))
        parts, pieces = check(new.tolist(), ctx.tolist(), heads, group, grid, whole=True)
        assert all(p[4] == -1 for p in pieces)
        if len(pieces) <= grid:
            assert sorted(p[0] for p in pieces) == list(range(len(pieces)))


def test_no_work():
    for new, ctx in (([0], [0]), ([0, 0], [5, 0]), ([3], [0])):
        check(new, ctx, 2, 4, 152)


def test_far_lengths():
    # a million keys and a long chunk: the root of the quadratic stays exact enough
    check([20000, 1, 16384], [1 << 20, 1 << 20, (1 << 20) + 5], 2, 8, 152)
    check([1 << 18], [1 << 21], 1, 3, 152)


def test_balance():
    """No CTA has more key tiles than its part of the line holds, plus one."""
    seqs, total, parts, pieces = plan([2048], [65049], 8, 4, 152)
    tiles = np.zeros(parts)
    for cta, _, t0, t1, _ in pieces:
        tiles[cta] += t1 - t0
    assert tiles.max() <= total / parts / KEYS + 1
