"""CPU pins of oracle/long_context.py by closed forms and by mistakes planted in it."""
import numpy as np
import pytest

from oracle import long_context as lc


def test_rope_keeps_lengths_and_relative_positions():
    rng = np.random.default_rng(0)
    inv = 10000.0 ** (-np.arange(16) / 16)
    q, k = rng.normal(size=(2, 5, 1, 40))
    for inter in (False, True):
        a = lc.rope(q, [3, 9, 20, 0, 7], inv, interleaved=inter)
        assert np.allclose((a[..., :32] ** 2).sum(-1), (q[..., :32] ** 2).sum(-1))
        assert np.array_equal(a[..., 32:], q[..., 32:]) and np.array_equal(a[3], q[3])
        # a product depends on the distance of the positions alone
        one = [(lc.rope(q, [p] * 5, inv, interleaved=inter) * lc.rope(k, [p - 4] * 5, inv, interleaved=inter)).sum(-1)
               for p in (4, 1000)]
        assert np.allclose(one[0], one[1])
    turned = lc.rope(np.array([[[1.0, 0.0]]]), [[1]], [np.pi / 2])
    assert np.allclose(turned, [[[0.0, 1.0]]])


def test_rope_axes_take_their_own_positions():
    inv = 0.1 * np.arange(1, 9)
    x = np.random.default_rng(1).normal(size=(3, 2, 16))
    pos = np.array([[1, 2, 3], [9, 9, 0]])
    both = lc.rope(x, pos, inv, axes=[0] * 4 + [1] * 4)
    a, b = lc.rope(x, pos[0], inv), lc.rope(x, pos[1], inv)
    first = [0, 1, 2, 3, 8, 9, 10, 11]
    assert np.array_equal(both[..., first], a[..., first])
    rest = [4, 5, 6, 7, 12, 13, 14, 15]
    assert np.array_equal(both[..., rest], b[..., rest])


def test_chunk_attention_is_causal():
    rng = np.random.default_rng(2)
    D, L, n = 8, 21, 6
    pool = rng.normal(size=(2, 4, 1, 16, D))
    tables, lens, off = np.array([[3, 1]]), [L], [0, n]
    q = rng.normal(size=(n, 2, D))
    out, _ = lc.chunk_attention(q, *pool, tables, lens, off, 0.3)
    changed = pool.copy()
    changed[:, 1, 0, 20 - 16] = np.nan                               # the last token: only the last row sees it
    again, _ = lc.chunk_attention(q, *changed, tables, lens, off, 0.3)
    assert np.array_equal(again[:5], out[:5]) and np.isnan(again[5]).all()
    # zero logits: the mean of what is seen
    flat, mag = lc.chunk_attention(0 * q, *pool, tables, lens, off, 0.3)
    v = lc.gather(pool[1], tables[0], L, 0)
    for i in range(n):
        assert np.allclose(flat[i, 0], v[:L - n + i + 1].mean(0)) and np.allclose(mag[i, 1], np.abs(v[:L - n + i + 1]).mean(0))
    # a context shorter than the chunk
    short, _ = lc.chunk_attention(q, *pool, tables, [4], off, 0.3)
    assert not short[:2].any() and np.allclose(short[2, 0], lc.gather(pool[1], tables[0], 1, 0)[0])


def test_bounds_bound_every_product():
    rng = np.random.default_rng(3)
    for n in (1, 5, 16):
        k = (rng.normal(size=(n, 64)) * np.exp(rng.normal(size=64))).astype(np.float32)
        code, s = lc.block_bounds(k)
        edge = code.astype(np.float64) * float(s)
        slack = 1e-6 * float(np.abs(k).max())
        assert (edge[0] >= k.max(0) - slack).all() and (edge[1] <= k.min(0) + slack).all()
        assert (edge[0] - k.max(0) < float(s) + slack).all()
        q = rng.normal(size=64)
        assert np.maximum(q * edge[0], q * edge[1]).sum() >= (k @ q).max() - 1e-3
        # planted: rounding to nearest would not bound
        near = np.rint(k.max(0) / s) * float(s)
        assert (near < k.max(0) - slack).any()
    code, s = lc.block_bounds(np.zeros((4, 64)))
    assert s == 0 and not code.any()
    code, s = lc.block_bounds(np.full((1, 64), np.nan))
    assert np.isinf(s) and (code[0] == 127).all() and (code[1] == -127).all()


@pytest.mark.parametrize("num", [4, 6])
def test_selection(num):
    D = 64
    bounds = np.zeros((10, 1, 2, D), np.int8)
    scales = np.full((10, 1), 0.5, np.float32)
    bounds[:, 0, 0, 0] = [0, 3, 9, 3, 3, 100, 3, 9, 0, 0]
    q = np.zeros((1, 1, D))
    q[0, 0, 0] = 2.0
    got = lc.select_blocks(q, bounds, scales, np.arange(10)[None], [150], num, 1, 1)
    assert got[0, 0].tolist() == {4: [0, 2, 5, 9], 6: [0, 1, 2, 5, 7, 9]}[num]    # equals: the lowest first
    got = lc.select_blocks(q, bounds, scales, np.arange(10)[None], [33], num, 1, 1)
    assert got[0, 0].tolist() == [0, 1, 2] + [-1] * (num - 3)
    scales[7] = np.inf
    assert 7 in lc.select_blocks(q, bounds, scales, np.arange(10)[None], [150], num, 1, 1)
    q[0, 0, 3] = np.nan                                               # no codes: the lowest blocks
    assert lc.select_blocks(q, bounds, np.full((10, 1), 0.5), np.arange(10)[None], [150], 4, 1, 1).tolist() == [[[0, 1, 2, 9]]]


def test_sparse_attention_over_all_blocks_is_attention():
    rng = np.random.default_rng(4)
    pool = rng.normal(size=(2, 6, 2, 16, 8))
    tables, lens = np.array([[5, 0, 3], [1, 2, -1]]), [40, 17]
    q = rng.normal(size=(2, 6, 8))
    full = np.array([[[0, 1, 2]] * 2, [[1, -1, 0]] * 2])
    out, _ = lc.sparse_attention(q, *pool, tables, lens, full, 0.4)
    ref, _ = lc.chunk_attention(q, *pool, tables, lens, [0, 1, 2], 0.4)
    assert np.allclose(out, ref)
    twice, _ = lc.sparse_attention(q, *pool, tables, lens, np.array([[[2, 2]] * 2, [[-1, -1]] * 2]), 0.4)
    once, _ = lc.sparse_attention(q, *pool, tables, lens, np.array([[[2, -1]] * 2, [[-1, -1]] * 2]), 0.4)
    assert np.allclose(twice[0], once[0]) and not twice[1].any()
