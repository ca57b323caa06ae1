"""4-bit KV cache in plain numpy: quantisation of a row, the tile's byte order,
append, and the values that a pool stands for (float64).

The format (one scale and one minimum per row, float16; codes 0..15; the byte
order within a tile) is this library's own; the pages only say that fewer bits
per value mean fewer bytes per token."""
from __future__ import annotations

import numpy as np

from . import widen

BLOCK = 16
F16_MAX = np.float32(65504.0)


def quantise_rows(x: np.ndarray):
    """Codes uint8 [..., D] and float16 pairs [..., 2] (scale, minimum) of rows
    of values [..., D]; every step in IEEE float32, as the contract says.  A row
    with a NaN: codes 0, scale 0, minimum NaN (0x7FFF)."""
    x = np.clip(np.asarray(x, np.float32), -F16_MAX, F16_MAX)
    bad = np.isnan(x).any(-1, keepdims=True)
    x = np.where(bad, np.float32(0), x)
    low = x.min(-1, keepdims=True).astype(np.float16)
    lowf = low.astype(np.float32)
    scale = ((x.max(-1, keepdims=True) - lowf) / np.float32(15)).astype(np.float16)
    sf = scale.astype(np.float32)
    inv = np.divide(np.float32(1), sf, out=np.zeros_like(sf), where=sf > 0)
    codes = np.clip(np.rint((x - lowf) * inv), 0, 15).astype(np.uint8)
    low = np.where(bad, np.uint16(0x7FFF), low.view(np.uint16)).view(np.float16)
    return codes, np.concatenate([scale, low], -1)


def code_byte(t: int, d: int, head_dim: int, is_v: bool):
    """(byte within the tile, shift) of the code of dim d of the token at offset t."""
    if not is_v:
        return t * (head_dim // 2) + d // 2, 4 * (d % 2)
    g = head_dim // 8
    at = (t // 8) * 4 * head_dim + (d // g) * 4 * g + (t // 2 % 4) * g + (d % g) // 4 * 4 + (t % 2) * 2 + d % 4 // 2
    return at, 4 * (d % 2)


def code_map(head_dim: int, is_v: bool):
    """code_byte of every (t, d): int arrays [16][D]."""
    m = np.array([[code_byte(t, d, head_dim, is_v) for d in range(head_dim)] for t in range(BLOCK)])
    return m[..., 0], m[..., 1]


def tiles(pool: np.ndarray) -> np.ndarray:
    nb, hkv = pool.shape[:2]
    return pool.reshape(nb, hkv, -1)


def head_dim_of(pool: np.ndarray) -> int:
    return 2 * (pool.shape[3] - 4)


def append_one(pool: np.ndarray, rows: np.ndarray, slots: np.ndarray, is_v: bool) -> np.ndarray:
    """A copy of pool uint8 [NB][Hkv][16][D/2 + 4] with rows [T][Hkv][D] (values)
    stored at their slots; negative slots skipped."""
    out = pool.copy()
    d = head_dim_of(pool)
    at, shift = code_map(d, is_v)
    codes, pairs = quantise_rows(rows)
    flat = tiles(out)
    slots = np.asarray(slots, np.int64)
    keep = np.flatnonzero(slots >= 0)
    blk, t = slots[keep] // BLOCK, slots[keep] % BLOCK     # distinct slots: distinct bytes
    for j in range(d):
        if j % 2 == 0:
            flat[blk, :, at[t, j]] = 0
        flat[blk, :, at[t, j]] |= codes[keep, :, j] << np.uint8(shift[0, j])
    for i in range(4):
        flat[blk, :, 8 * d + 4 * t + i] = np.ascontiguousarray(pairs[keep]).view(np.uint8)[..., i]
    return out


def kv_append_int4(k_pool, v_pool, k_bits, v_bits, slots, dtype: str):
    """Both pools after the append of k_bits / v_bits [T][Hkv][D] (16-bit patterns of dtype)."""
    return (append_one(k_pool, widen(k_bits, dtype).astype(np.float32), slots, False),
            append_one(v_pool, widen(v_bits, dtype).astype(np.float32), slots, True))


def values(pool: np.ndarray, is_v: bool) -> np.ndarray:
    """What a pool stands for: float64 [NB][Hkv][16][D]."""
    d = head_dim_of(pool)
    at, shift = code_map(d, is_v)
    flat = tiles(pool)
    codes = (flat[:, :, at] >> shift.astype(np.uint8)) & 15
    pairs = np.ascontiguousarray(flat[:, :, 8 * d:]).view(np.float16).reshape(*flat.shape[:2], BLOCK, 2)
    with np.errstate(invalid="ignore"):
        return codes.astype(np.float64) * pairs[..., :1].astype(np.float64) + pairs[..., 1:].astype(np.float64)


def decode_attention(q, k_pool, v_pool, tables, lens, scale):
    """float64 [B][Hq][D] over 4-bit pools; q float64 [B][Hq][D]."""
    B, H, D = q.shape
    hk = k_pool.shape[1]
    g = H // hk
    out = np.zeros((B, H, D))
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        ids = np.asarray(tables[b, :-(-n // BLOCK)], np.int64)
        K, V = values(k_pool[ids], False), values(v_pool[ids], True)
        for h in range(hk):
            k, v = K[:, h].reshape(-1, D)[:n], V[:, h].reshape(-1, D)[:n]
            s = q[b, h * g:(h + 1) * g] @ k.T * scale
            p = np.exp(s - s.max(-1, keepdims=True))
            out[b, h * g:(h + 1) * g] = (p @ v) / p.sum(-1, keepdims=True)
    return out
