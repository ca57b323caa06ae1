"""CPU model of the 4-bit decode kernel's index arithmetic: the partition with
its share rule, the cutting of windows into stages, and the merges' search for
the pieces the decode kernel leaves (constants read from the kernel sources)."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_26_gb300", "csrc")
KERNELS = open(os.path.join(CSRC, "paged_kv_kernels.cuh")).read()
INT4 = open(os.path.join(CSRC, "decode_int4.cuh")).read()


def const(text, name):
    return int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))


UNIT, NB, WARPS = const(INT4, "kInt4ShareUnit"), const(INT4, "kBlocksPerStage"), const(INT4, "kWarps")
MIN2, MIN3, MIN4 = (const(KERNELS, n) for n in ("kMinDynamicShare", "kThreeChunkShare", "kFourChunkShare"))


class Partition:
    def __init__(self, total, nwarps, units, unit=UNIT):
        self.total, self.nwarps = total, nwarps
        r = -(-total // nwarps) if total > 0 else 1
        if total > 0 and unit > 1:
            r = max(r, min(2 * unit, total // units // 32))
            if unit < r < 2 * unit:
                r = 2 * unit
        self.R = r
        self.n = 0 if r < MIN2 * unit else 2 if r < MIN3 * unit else 3 if r < MIN4 * unit else 4
        self.cum = {0: [0], 2: [0, 8, 10], 3: [0, 7, 9, 10], 4: [0, 4, 7, 9, 10]}[self.n]

    def head(self, w):
        s = min(self.total, w * self.R)
        n = min(self.total, (w + 1) * self.R) - s
        return s, s + (n if self.n == 0 else n * 17 // 20 if self.n == 2 else n * 4 // 5)

    def chunk(self, k, w):
        he = self.head(w)[1]
        tail = min(self.total, (w + 1) * self.R) - he
        return he + tail * self.cum[k] // 10, he + tail * self.cum[k + 1] // 10

    def segments(self):
        out = [(w, *self.head(w)) for w in range(self.nwarps)]
        return out + [(self.nwarps + k * self.nwarps + w, *self.chunk(k, w)) for k in range(self.n)
                      for w in range(self.nwarps)]

    def segment_of(self, p):
        w = p // self.R
        s, e = self.head(w)
        if p < e:
            return s, e
        for k in range(self.n):
            s, e = self.chunk(k, w)
            if p < e:
                return s, e
        raise AssertionError


def batches():
    rng = np.random.default_rng(0)
    yield [7], 2, 152
    yield [1], 1, 152
    yield [128] * 8, 8, 152
    yield [512], 8, 152
    yield [2048] * 8, 8, 152
    yield list(rng.integers(32, 257, 64)), 8, 152
    yield [5000, 1, 0, 3, 700], 3, 152
    yield list(rng.integers(0, 40, 300)), 5, 152
    yield list(rng.integers(500, 2500, 12)), 8, 20          # shares with dynamic tails
    yield list(rng.integers(500, 2500, 40)), 8, 12
    yield list(rng.integers(2000, 9000, 40)), 8, 30


@pytest.mark.parametrize("case", range(11))
def test_every_block_once_and_every_piece_found(case):
    nbs, hkv, sms = list(batches())[case]
    B = len(nbs)
    P = np.concatenate([[0], np.cumsum(nbs)]).astype(int)
    part = Partition(hkv * int(P[-1]), sms * WARPS, B * hkv)
    seen = np.zeros(part.total, int)
    units = [(hkv * int(P[b]) + k * nbs[b], nbs[b]) for b in range(B) for k in range(hkv)]
    starts = np.array([u for u, _ in units])
    wrote, direct = {}, set()
    for sid, s, e in part.segments():
        seen[s:e] += 1
        p, first = s, True
        while p < e:                                        # the units of this segment, in order
            i = int(np.searchsorted(starts, p, side="right")) - 1
            while units[i][1] == 0:
                i -= 1
            U, nb = units[i]
            q = min(e, U + nb)
            if p == U and q == U + nb:
                direct.add(i)
            else:
                wrote.setdefault(i, set()).add(sid * 2 + (0 if first else 1))
            p, first = q, False
    assert (seen == 1).all()
    per = 1 + part.n
    for i, (U, nb) in enumerate(units):                     # merge_units_kernel's plan and gather
        if nb == 0:
            continue
        w0, w1 = U // part.R, (U + nb - 1) // part.R
        if part.n == 0:
            ncand = w1 - w0 + 1 if w1 > w0 else 0
        else:
            ncand = (w1 - w0 + 1) * per if part.segment_of(U)[1] < U + nb else 0
        found = set()
        for c in range(ncand):
            w, k = (w0 + c, 0) if part.n == 0 else (w0 + c // per, c % per)
            s, e = part.head(w) if k == 0 else part.chunk(k - 1, w)
            sid = w if k == 0 else part.nwarps + (k - 1) * part.nwarps + w
            if e <= s or e <= U or s >= U + nb:
                continue
            found.add(sid * 2 + (1 if U > s else 0))
        assert found == wrote.get(i, set()), (i, U, nb)
        assert (ncand == 0) == (i in direct)


@pytest.mark.parametrize("append", [False, True])
def test_windows_are_cut_into_whole_stages(append):
    """fill_window: the stages of random windows cover their blocks in order, stay
    within one unit and the ring's size, and leave room for the appended rows."""
    rng = np.random.default_rng(1)
    for _ in range(300):
        ctx = rng.integers(1, 200, 12)
        nbs = -(-ctx // 16)
        flat = [(u, j) for u in range(12) for j in range(nbs[u])]
        s = int(rng.integers(0, len(flat)))
        e = int(rng.integers(s + 1, min(len(flat), s + 60) + 1))
        ip, blocks, left = s, [], {}
        while ip < e:
            win = flat[ip:min(e, ip + 32)]
            n = len(win)
            runs = [i for i in range(n) if i == 0 or win[i][1] == 0]
            pos = [i - max(r for r in runs if r <= i) for i in range(n)]
            firsts = [i for i in range(n) if pos[i] % NB == 0 or
                      (append and win[i][1] == nbs[win[i][0]] - 1 and pos[i] % NB == NB - 1)]
            for a, f in enumerate(firsts):
                count = (firsts[a + 1] if a + 1 < len(firsts) else n) - f
                u, j = win[f]
                assert 1 <= count <= NB and all(w == (u, j + k) for k, w in enumerate(win[f:f + count]))
                valid = min(16 * count, int(ctx[u]) - 16 * j)
                assert 16 * (count - 1) < valid <= 16 * count
                end = j + count == nbs[u]
                if append and end:
                    assert count < NB                       # the new rows take the last block's place
                    assert (valid - 1) % 16 == (ctx[u] - 1) % 16
                left[u] = left.get(u, 0) + valid
                blocks += win[f:f + count]
            ip += n
        assert blocks == flat[s:e]
