"""float64 definitions of rotary positions, chunk attention and block-sparse decode
(numpy, CPU; test infrastructure).  Pools and rows are arrays of values here:
K and V pools [num_blocks][Hkv][16][D]."""
import numpy as np

BLOCK = 16


def rope(x, positions, inv_freq, axes=None, interleaved=False, factor=1.0):
    """x [T][H][D] turned to positions [axes][T]; frequency f takes positions[axes[f]]."""
    x = np.asarray(x, np.float64)
    pos = np.atleast_2d(np.asarray(positions, np.float64))
    n = len(inv_freq)
    angle = np.stack([pos[0 if axes is None else axes[f]] * inv_freq[f] for f in range(n)], -1)[:, None]
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    out = x.copy()
    out[..., i] = x[..., i] * c - x[..., j] * s
    out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def gather(pool, table, n, kvh):
    """The first n tokens' rows of KV head kvh, [n][D]."""
    ids = np.asarray(table[:-(-n // BLOCK)], np.int64)
    return np.asarray(pool[ids, kvh], np.float64).reshape(-1, pool.shape[-1])[:n]


def attend(q, k, v, seen, scale):
    """Rows q [n][D] over keys k, v [m][D]; seen [n][m] tells what a row attends to.
    Returns the outputs and the weighted means of |v| (what rounding a weight acts on).
    A row that sees nothing is zero, one whose logits are all -infinity NaN; values that
    no row sees do not matter."""
    any_seen = seen.any(0)
    k = np.where(any_seen[:, None], k, 0.0)
    with np.errstate(invalid="ignore"):
        s = (q @ k.T) * scale
    s = np.where(seen, s, -np.inf)
    top = s.max(-1, initial=-np.inf, keepdims=True)
    with np.errstate(invalid="ignore"):
        p = np.where(seen, np.exp(s - np.where(np.isneginf(top), 0.0, top)), 0.0)
        total = p.sum(-1, keepdims=True)
        p = np.divide(p, total, out=np.zeros_like(p), where=seen.any(-1, keepdims=True))
    bad = ~np.isfinite(v) & any_seen[:, None]
    vf = np.where(np.isfinite(v), v, 0.0)
    out, mag = p @ vf, p @ np.abs(vf)
    for t in np.flatnonzero(bad.any(1)):          # a value that is not finite reaches the rows that see it
        rows = np.flatnonzero(seen[:, t])
        with np.errstate(invalid="ignore"):
            out[rows] += np.where(bad[t], v[t], 0.0) * p[rows, t][:, None]
    return out, mag


def chunk_attention(q, k_pool, v_pool, tables, lens, offsets, scale):
    """Outputs [T][Hq][D] (NaN in rows outside the offsets) and mean |v|."""
    T, Hq, D = q.shape
    Hk = k_pool.shape[1]
    g = Hq // Hk
    out, mag = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    for b, L in enumerate(int(x) for x in lens):
        r0, n = int(offsets[b]), int(offsets[b + 1] - offsets[b])
        if n <= 0:
            continue
        seen = np.arange(L)[None] <= (L - n + np.arange(n))[:, None]
        for h in range(Hq):
            k, v = gather(k_pool, tables[b], L, h // g), gather(v_pool, tables[b], L, h // g)
            out[r0:r0 + n, h], mag[r0:r0 + n, h] = attend(np.asarray(q[r0:r0 + n, h], np.float64), k, v, seen, scale)
    return out, mag


def block_bounds(k):
    """Codes [2][D] (int8: upper, lower) and scale of one block's valid keys [n][D], in float32."""
    k = np.asarray(k, np.float32)
    if not np.isfinite(k).all():
        return np.stack([np.full(k.shape[1], 127, np.int8), np.full(k.shape[1], -127, np.int8)]), np.float32(np.inf)
    hi, lo = k.max(0), k.min(0)
    scale = np.float32(np.maximum(np.abs(hi), np.abs(lo)).max() * (np.float32(1) / np.float32(127)))
    if not scale > 0:
        return np.zeros((2, k.shape[1]), np.int8), scale
    return np.stack([np.clip(np.ceil(hi / scale), -127, 127), np.clip(np.floor(lo / scale), -127, 127)]).astype(np.int8), scale


def update_bounds(k_pool, tables, lens, offsets, bounds, scales):
    """bounds / scales after the blocks with new tokens (offsets None: one each) are made anew."""
    bounds, scales = bounds.copy(), scales.copy()
    for b, L in enumerate(int(x) for x in lens):
        n = 1 if offsets is None else int(offsets[b + 1] - offsets[b])
        if n <= 0 or L == 0:
            continue
        for j in range(max(L - n, 0) // BLOCK, -(-L // BLOCK)):
            p = int(tables[b, j])
            for x in range(k_pool.shape[1]):
                bounds[p, x], scales[p, x] = block_bounds(k_pool[p, x, :min(BLOCK, L - j * BLOCK)])
    return bounds, scales


def block_scores(q, bounds, scales):
    """q [g][D] of one group, bounds [n][2][D], scales [n]: float32 scores [n]."""
    q = np.asarray(q, np.float32)
    best = np.full(len(bounds), -np.inf, np.float32)
    one = np.float32(1) / np.float32(127)
    for row in q:
        r = np.float32(np.abs(row).max() * one)      # an infinity or NaN where the row holds one: its scores are NaN
        c = np.rint(row / r).astype(np.int64) if r > 0 and np.isfinite(r) else np.zeros(q.shape[1], np.int64)
        e = bounds.astype(np.int64)
        dot = np.maximum(c * e[:, 0], c * e[:, 1]).sum(-1)
        with np.errstate(invalid="ignore"):
            s = dot.astype(np.float32) * scales.astype(np.float32) * r
        best = np.maximum(best, np.where(np.isnan(s), np.float32(np.inf), s))
    return best


def select_blocks(q, bounds, scales, tables, lens, num, sink, recent):
    B, Hq, _ = q.shape
    Hk = bounds.shape[1]
    g = Hq // Hk
    out = np.full((B, Hk, num), -1, np.int32)
    for b, L in enumerate(int(x) for x in lens):
        nb = -(-L // BLOCK)
        ids = np.asarray(tables[b, :nb], np.int64)
        keep = set(range(min(sink, nb))) | set(range(max(0, nb - recent), nb))
        for x in range(Hk):
            score = block_scores(q[b, x * g:(x + 1) * g], bounds[ids, x], scales[ids, x])
            rest = sorted((j for j in range(nb) if j not in keep), key=lambda j: (-score[j], j))
            some = sorted((sorted(keep) + rest)[:num]) if nb > num else list(range(nb))
            out[b, x, :len(some)] = some
    return out


def sparse_attention(q, k_pool, v_pool, tables, lens, selected, scale):
    B, Hq, D = q.shape
    Hk = k_pool.shape[1]
    g = Hq // Hk
    out, mag = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b, L in enumerate(int(x) for x in lens):
        for x in range(Hk):
            pos = [p for j in selected[b, x] if 0 <= j < -(-L // BLOCK) for p in range(j * BLOCK, min((j + 1) * BLOCK, L))]
            if not pos:
                continue
            pos = np.asarray(pos)
            ids = np.asarray(tables[b], np.int64)[pos // BLOCK]
            k, v = (np.asarray(p[ids, x, pos % BLOCK], np.float64) for p in (k_pool, v_pool))
            h = slice(x * g, (x + 1) * g)
            out[b, h], mag[b, h] = attend(np.asarray(q[b, h], np.float64), k, v, np.ones((g, len(pos)), bool), scale)
    return out, mag
