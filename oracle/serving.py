"""Plain Python of the GPU block tables and of draft verification: a stack of
free blocks walked token by token, and whole-number sums of any length."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

BLOCK = 16


def resize_tables(lens, new_lens, tables, free, num_free):
    """(slots, offsets, tables, free, num_free) after every sequence went from
    lens[b] to new_lens[b] tokens, or None if there are too few blocks.  Given
    blocks go on the stack first, last (sequence, block) first; then taken ones
    come off its top, first (sequence, position) first."""
    tables = np.array(tables)
    free = list(map(int, free))
    stack = free[:num_free]
    given = [int(tables[b, j]) for b, (o, n) in enumerate(zip(lens, new_lens))
             for j in range(-(-int(n) // BLOCK), -(-int(o) // BLOCK))]
    stack += given[::-1]
    if len(stack) > len(free):
        raise ValueError("more blocks given than the list can hold")
    slots, offsets = [], [0]
    for b, (o, n) in enumerate(zip(lens, new_lens)):
        for pos in range(int(o), int(n)):
            if pos % BLOCK == 0:
                if not stack:
                    return None
                tables[b, pos // BLOCK] = stack.pop()
            slots.append(int(tables[b, pos // BLOCK]) * BLOCK + pos % BLOCK)
        offsets.append(len(slots))
    out = list(free)
    out[:len(stack)] = stack
    return slots, offsets, tables, out, len(stack)


def weight(p: float) -> int:
    """A probability as a whole number of 2^-40, half to even."""
    if not p > 0:
        return 0
    return round(Fraction(min(float(p), 1.0)) * (1 << 40))  # Python rounds half to even


def draw(weights, u: float):
    """Lowest index whose running sum exceeds floor(total * U / 2^30)."""
    total = sum(weights)
    if total == 0:
        return -1
    u30 = 0 if not u > 0 else min(math.floor(Fraction(min(float(u), 1.0)) * (1 << 30)), (1 << 30) - 1)
    goal, run = total * u30 >> 30, 0
    for v, w in enumerate(weights):
        run += w
        if run > goal:
            return v
    raise AssertionError("unreachable")


def verify_one(target, draft, tokens, n, accept_u, sample_u):
    """(accepted, drawn token) of one sequence: target [K + 1][V] and draft
    [K][V] (or None) of floats, n of its K drafts in use."""
    vocab = len(target[0])
    for i in range(n):
        x = int(tokens[i])
        q = 1.0 if draft is None else float(draft[i][x])
        if 0 <= x < vocab and Fraction(float(accept_u[i])) * Fraction(q) < Fraction(float(target[i][x])):
            continue
        p = [weight(v) for v in target[i]]
        if draft is not None:
            rest = [max(a - weight(c), 0) for a, c in zip(p, draft[i])]
        else:
            rest = [max(a - (1 << 40), 0) if v == x else a for v, a in enumerate(p)]
        return i, draw(rest if any(rest) else p, sample_u)
    return n, draw([weight(v) for v in target[n]], sample_u)
