"""CPU model of the 4-bit decode kernel's index arithmetic: the shares, the
cutting of windows into stages, and where the merge finds the pieces that the
decode kernel leaves (constants read from the kernel source)."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_26_gb300", "csrc")
INT4 = open(os.path.join(CSRC, "decode_int4.cuh")).read()


def const(text, name):
    return int(re.search(rf"constexpr int {name} = (\d+);", text).group(1))


FEW, NB, WARPS = const(INT4, "kFew"), const(INT4, "kBlocksPerStage"), const(INT4, "kWarps")


class Shares:
    def __init__(self, total, nwarps, units):
        self.total, self.R = total, 1
        if total > 0:
            self.R = max(-(-total // nwarps), min(FEW, total // units // 32), total // units // 256)
            if FEW // 2 < self.R < FEW:
                self.R = FEW

    def start(self, w):
        return min(self.total, w * self.R)


def batches():
    rng = np.random.default_rng(0)
    yield [7], 2, 152
    yield [1], 1, 152
    yield [128] * 8, 8, 152
    yield [512], 8, 152
    yield [8192], 1, 152
    yield [2048] * 8, 8, 152
    yield list(rng.integers(32, 257, 64)), 8, 152
    yield [5000, 1, 0, 3, 700], 3, 152
    yield list(rng.integers(0, 40, 300)), 5, 152
    yield list(rng.integers(500, 2500, 12)), 8, 20
    yield list(rng.integers(500, 2500, 40)), 8, 12
    yield list(rng.integers(2000, 9000, 40)), 8, 30


@pytest.mark.parametrize("case", range(12))
def test_every_block_once_and_every_piece_found(case):
    nbs, hkv, sms = list(batches())[case]
    B, nwarps = len(nbs), sms * WARPS
    P = np.concatenate([[0], np.cumsum(nbs)]).astype(int)
    part = Shares(hkv * int(P[-1]), nwarps, B * hkv)
    seen = np.zeros(part.total, int)
    units = [(hkv * int(P[b]) + k * nbs[b], nbs[b]) for b in range(B) for k in range(hkv)]
    starts = np.array([u for u, _ in units])
    wrote, direct = {}, set()
    for w in range(nwarps):
        s, e = part.start(w), part.start(w + 1)
        seen[s:e] += 1
        p, first = s, True
        while p < e:                                        # the units of this share, in order
            i = int(np.searchsorted(starts, p, side="right")) - 1
            while units[i][1] == 0:
                i -= 1
            U, nb = units[i]
            q = min(e, U + nb)
            if p == U and q == U + nb:
                direct.add(i)
            else:
                wrote.setdefault(i, []).append(w * 2 + (0 if first else 1))
            p, first = q, False
    assert (seen == 1).all()
    for i, (U, nb) in enumerate(units):                     # UnitPieces and merge_int4_kernel's row()
        w = U // part.R
        n = (U + nb - 1) // part.R - w + 1 if nb > 0 else 1
        first, count = 2 * w + (U > w * part.R), n if n > 1 else 0
        assert [first if p == 0 else first // 2 * 2 + 2 * p for p in range(count)] == wrote.get(i, [])
        assert (count == 0) == (nb == 0 or i in direct)


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
