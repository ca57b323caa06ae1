"""GPU: bounds of blocks and the selection exactly, attention over selected blocks
against float64 (bound: long_context_helpers.tolerance; bf16 weights enter as two
terms, good to 2^-16, fp16 ones as one)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, hide_tails, i32, paged, rand, tolerance
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
BITS = {"fp16": 11, "bf16": 16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def keys(nb, hk, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp(torch.randn(hk, 1, d, generator=g))
    return ((torch.randn(nb, hk, 16, d, generator=g) + torch.randn(nb, hk, 1, d, generator=g)) * spread).to(DT[dtype])


def equal_bounds(bounds, scales, ref):
    assert np.array_equal(bounds.cpu().numpy(), ref[0]) and np.array_equal(scales.cpu().numpy(), ref[1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hk", [(64, 1), (64, 5), (128, 3), (128, 8)])
def test_bounds(dtype, d, hk):
    new = [0, 1, 16, 5, 33, 200, 1, 0, 7, 40]
    lens = [0, 1, 16, 21, 64, 200, 300, 70, 7, 15]                  # the last: more new tokens than context
    tables, nb = paged(lens, 1)
    kp = keys(nb, hk, d, dtype, 2)
    kp[tables[4, 3], 0, 2, 5] = float("inf")
    kp[tables[5, 0], hk - 1, 15, 0] = float("nan")
    kp[tables[5, 1], 0] = 0
    kp[tables[5, 2], 0] *= 0
    kp[tables[5, 3], 0] = -0.0
    kp[tables[5, 4], 0] = torch.tensor(6e-8, dtype=DT[dtype])       # the smallest values
    kp = hide_tails(kp, tables, lens)
    off = np.concatenate([[0], np.cumsum(new)])
    rng = np.random.default_rng(0)
    b0, s0 = rng.integers(-127, 128, (nb, hk, 2, d)).astype(np.int8), rng.random((nb, hk)).astype(np.float32)
    for offsets, many in ((off, int(off[-1])), (off, int(off[-1]) + 1000), (off + 37, int(off[-1]) + 37), (None, None)):
        bounds, scales = torch.from_numpy(b0).to(DEV, copy=True), torch.from_numpy(s0).to(DEV, copy=True)
        pkv.paged_kv_update_bounds(kp.to(DEV), i32(tables), i32(lens), bounds, scales,
                                   q_offsets=None if offsets is None else i32(offsets), num_tokens=many)
        pkv.paged_kv_check_status()
        equal_bounds(bounds, scales, lc.update_bounds(kp.float().numpy(), tables, lens, offsets, b0, s0))


def test_bounds_of_many_sequences_and_bad_arguments():
    rng = np.random.default_rng(1)
    new = rng.integers(0, 40, 3000)
    lens = new + rng.integers(0, 30, 3000)
    tables, nb = paged(lens, 3)
    kp = keys(nb, 2, 64, "bf16", 4)
    off = np.concatenate([[0], np.cumsum(new)])
    bounds, scales = torch.zeros(nb, 2, 2, 64, dtype=torch.int8, device=DEV), torch.zeros(nb, 2, device=DEV)
    pkv.paged_kv_update_bounds(kp.to(DEV), i32(tables), i32(lens), bounds, scales, i32(off), int(off[-1]))
    pkv.paged_kv_check_status()
    ref = lc.update_bounds(kp.float().numpy(), tables, lens, off, np.zeros((nb, 2, 2, 64), np.int8),
                           np.zeros((nb, 2), np.float32))
    equal_bounds(bounds, scales, ref)

    def flagged(t, l, o, many):
        pkv.paged_kv_update_bounds(kp.to(DEV), i32(t), i32(l), bounds, scales, None if o is None else i32(o), many)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == -6

    bad = tables[:2].copy()
    lens2 = [20, 20]
    bad = np.full((2, 2), -1, np.int32)
    flagged(bad, lens2, None, None)
    bad[:] = nb
    flagged(bad, lens2, [0, 5, 25], 25)
    good = np.array([[0, 1], [2, 3]], np.int32)
    flagged(good, [40, 20], None, None)              # longer than its table
    flagged(good, lens2, [0, 9, 4], 9)
    flagged(good, lens2, [0, 9, 40], 20)             # past num_tokens
    flagged(good, lens2, [-3, 9, 12], 20)
    equal_bounds(bounds[4:], scales[4:], (ref[0][4:], ref[1][4:]))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (2, 1), (6, 2), (4, 1), (10, 2), (8, 1)])
def test_selection_exact(dtype, d, hq, hk):
    lens = [0, 1, 16, 17, 330, 1000, 4111, 5000]
    tables, nb = paged(lens, 5)
    rng = np.random.default_rng(hq)
    bounds = np.sort(rng.integers(-127, 128, (nb, hk, 2, d)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.choice(np.float32([0.25, 0.5, 1e-3, 0.0]), (nb, hk))     # equal scores occur
    bounds[rng.random(nb) < 0.4] = bounds[0]
    scales[tables[5, 7], 0] = np.inf
    scales[tables[5, 9], 0] = np.inf
    q = rand((len(lens), hq, d), DT[dtype], 6, 3.0)
    q[4, 0] = 0.0
    q[6, hq - 1, 3] = float("nan")
    for num, sink, recent in ((1, 0, 1), (7, 1, 2), (64, 3, 4), (500, 0, 1), (6, 3, 3)):
        got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                      i32(tables), i32(lens), num, sink, recent)
        pkv.paged_kv_check_status()
        ref = lc.select_blocks(q.float().numpy(), bounds, scales, tables, lens, num, sink, recent)
        assert np.array_equal(got.cpu().numpy(), ref), (num, sink, recent)


@pytest.mark.parametrize("blocks", [32768, 32769, 70000])
def test_selection_of_very_long_contexts(blocks):
    """More keys than the selection holds in shared memory."""
    rng = np.random.default_rng(blocks)
    nb = 500
    tables = rng.integers(0, nb, (1, blocks)).astype(np.int32)
    bounds = np.sort(rng.integers(-127, 128, (nb, 1, 2, 64)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.random((nb, 1)).astype(np.float32)
    q = rand((1, 3, 64), torch.bfloat16, 1)
    lens = [blocks * 16 - 3]
    got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                  i32(tables), i32(lens), 300, 2, 3)
    pkv.paged_kv_check_status()
    # scores by block of the pool, then the rule
    score = lc.block_scores(q[0].float().numpy(), bounds[:, 0], scales[:, 0])[tables[0]]
    rest = np.arange(2, blocks - 3)
    best = rest[np.lexsort((rest, -score[rest]))][:295]
    want = np.sort(np.concatenate([[0, 1], blocks - 3 + np.arange(3), best]))
    assert np.array_equal(got.cpu().numpy()[0, 0], want)


@pytest.mark.parametrize("width,blocks", [(256, 256), (256, 33), (257, 257), (2048, 2048), (2049, 2049), (2048, 129), (8192, 8192), (8193, 8192),
                                          (8193, 8193), (9000, 1500), (40000, 700)])
@pytest.mark.parametrize("pool", [400, 12000])
def test_selection_at_the_borders_of_its_forms(width, blocks, pool):
    """Tables and contexts on either side of what one form of the choice holds, with many
    equal scores (few blocks in the pool) and with hardly any."""
    rng = np.random.default_rng(width + blocks)
    tables = np.full((2, width), -1, np.int32)
    lens = [blocks * 16, blocks * 16 - 17]
    bounds = np.sort(rng.integers(-127, 128, (pool, 2, 2, 64)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.random((pool, 2)).astype(np.float32)
    for b, n in enumerate(lens):
        tables[b, :-(-n // 16)] = rng.permutation(max(pool, blocks))[:-(-n // 16)] % pool
    q = rand((2, 10, 64), torch.bfloat16, 1)
    for num in (1, 60, 128):
        got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                      i32(tables), i32(lens), num, 0, 1)
        pkv.paged_kv_check_status()
        for b, n in enumerate(lens):
            n = -(-n // 16)
            for h in range(2):
                score = lc.block_scores(q[b, 5 * h:5 * h + 5].float().numpy(), bounds[:, h], scales[:, h])[tables[b, :n]]
                best = np.lexsort((np.arange(n - 1), -score[:n - 1]))[:num - 1]
                want = np.sort(np.append(best, n - 1))
                assert np.array_equal(got[b, h, :min(num, n)].cpu().numpy(), want[:n]), (b, h, num)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,seqs", [(1, 1, 304), (1, 1, 305), (6, 2, 152), (8, 2, 153), (16, 2, 150), (40, 8, 60), (5, 5, 3)])
def test_selection_in_one_and_two_launches(dtype, d, hq, hk, seqs):
    """Short tables of few and of more sequences, all lengths up to the table's."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 256 * 16 + 1, seqs)
    lens[:3] = (256 * 16, 0, 255 * 16 + 1)
    nb = 300
    tables = rng.integers(0, nb, (seqs, 256)).astype(np.int32)
    bounds = np.sort(rng.integers(-127, 128, (nb, hk, 2, d)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.random((nb, hk)).astype(np.float32)
    q = rand((seqs, hq, d), DT[dtype], 6)
    for num, sink, recent in ((20, 1, 2), (255, 0, 1)):
        got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                      i32(tables), i32(lens), num, sink, recent)
        pkv.paged_kv_check_status()
        ref = lc.select_blocks(q.float().numpy(), bounds, scales, tables, lens, num, sink, recent)
        assert np.array_equal(got.cpu().numpy(), ref), (num, sink, recent)


@pytest.mark.parametrize("seqs,hq,hk,width,num", [(70, 16, 8, 1000, 100), (600, 8, 8, 300, 40), (64, 40, 8, 2500, 64)])
def test_selection_of_many_long_tables(seqs, hq, hk, width, num):
    """More ranges of blocks than CTAs."""
    rng = np.random.default_rng(width)
    lens = rng.integers(0, width * 16 + 1, seqs)
    lens[:4] = (width * 16, 0, width * 16 - 15, 130 * 16)
    nb = 300
    tables = rng.integers(0, nb, (seqs, width)).astype(np.int32)
    bounds = np.sort(rng.integers(-127, 128, (nb, hk, 2, 128)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.random((nb, hk)).astype(np.float32)
    q = rand((seqs, hq, 128), torch.bfloat16, 6)
    got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                  i32(tables), i32(lens), num, 0, 1).cpu().numpy()
    pkv.paged_kv_check_status()
    g = hq // hk
    for b, length in enumerate(lens):
        n = -(-int(length) // 16)
        for h in range(hk):
            score = lc.block_scores(q[b, g * h:g * h + g].float().numpy(), bounds[:, h], scales[:, h])[tables[b, :n]]
            best = np.lexsort((np.arange(n - 1), -score[:n - 1]))[:num - 1] if n else np.empty(0, int)
            want = np.full(num, -1)
            want[:min(n, num)] = np.sort(np.append(best, n - 1))[:n] if n else []
            assert np.array_equal(got[b, h], want), (b, h)


def test_selection_flags_and_buffers():
    lens = [400, 30]
    tables, nb = paged(lens, 0)
    bounds, scales = torch.zeros(nb, 1, 2, 64, dtype=torch.int8, device=DEV), torch.ones(nb, 1, device=DEV)
    q = rand((2, 2, 64), torch.float16, 0).to(DEV)
    sel = torch.full((2, 1, 5), 9, dtype=torch.int32, device=DEV)
    need = int(tables.shape[1]) * 2 * 4 + 1024
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    got = pkv.paged_select_blocks(q, bounds, scales, i32(tables), i32(lens), 5, selected=sel, workspace=ws)
    assert got is sel and sel.tolist() == [[[0, 1, 2, 3, 24]], [[0, 1, -1, -1, -1]]]
    # no more blocks than selected: neither scores nor a workspace
    assert pkv.paged_select_blocks(q, bounds, scales, i32(tables), i32(lens), 25).tolist() == [[list(range(25))],
                                                                                           [[0, 1] + [-1] * 23]]
    bad = tables.copy()
    bad[0, 4] = nb
    pkv.paged_select_blocks(q, bounds, scales, i32(bad), i32(lens), 5)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_check_status()
    pkv.paged_select_blocks(q, bounds, scales, i32(tables), i32([401, 30]), 5)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_check_status()
    assert pkv.paged_select_blocks(q[:0], bounds, scales, i32(tables[:0]), i32([]), 5).shape == (0, 1, 5)


def attend(q, kp, vp, tables, lens, sel, scale, dtype, **kw):
    out = pkv.paged_decode_attention_sparse(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32(lens), i32(sel), scale, **kw)
    ref, mag = lc.sparse_attention(f64(q), f64(kp), f64(vp), tables, lens, sel, scale)
    tol = tolerance(ref, mag, DT[dtype], f64(q), f64(kp), f64(vp), scale, 16 * sel.shape[2], BITS[dtype])
    assert_within(f64(out), ref, tol)
    return out


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,num", [(1, 1, 1), (6, 2, 3), (8, 1, 17), (5, 5, 40), (16, 2, 300), (7, 1, 600)])
def test_attention(dtype, d, hq, hk, num):
    lens = [0, 1, 16, 37, 700, 3001]
    tables, nb = paged(lens, 2)
    kp, vp = (hide_tails(x, tables, lens) for x in (keys(nb, hk, d, dtype, 3), rand((nb, hk, 16, d), DT[dtype], 4)))
    q = rand((len(lens), hq, d), DT[dtype], 5)
    rng = np.random.default_rng(num)
    sel = np.full((len(lens), hk, num), -1, np.int32)
    for b, n in enumerate(lens):
        blocks = -(-n // 16)
        for x in range(hk):
            some = rng.permutation(blocks)[:num]                    # any order, -1 among them
            at = np.sort(rng.permutation(num)[:len(some)])
            sel[b, x, at] = some
    attend(q, kp, vp, tables, lens, sel, 0.3 * d ** -0.5, dtype)
    pkv.paged_kv_check_status()


def test_attention_lists():
    lens = [100, 40]
    tables, nb = paged(lens, 1)
    kp, vp, q = keys(nb, 2, 64, "bf16", 1), rand((nb, 2, 16, 64), torch.bfloat16, 2), rand((2, 4, 64), torch.bfloat16, 3)
    sel = np.array([[[0, 0, 5], [6, -1, 6]], [[-1] * 3, [2, 1, -7]]], np.int32)   # twice the same; none; negatives
    out = attend(q, kp, vp, tables, lens, sel, 0.125, "bf16")
    assert not out[1, :2].any()
    pkv.paged_kv_check_status()
    sel[0, 0, 1] = 7                                                               # behind the context: passed over
    attend(q, kp, vp, tables, lens, sel, -0.2, "bf16")
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_kv_check_status()
    assert e.value.code == -6
    out = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    pkv.paged_decode_attention_sparse(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32(lens),
                                      i32(np.zeros((2, 2, 0))), 0.125, out=out)
    assert not out.any()
    bad = tables.copy()
    bad[0, 5] = -1
    pkv.paged_decode_attention_sparse(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(bad), i32(lens), i32([[[5]] * 2] * 2), 0.1)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_check_status()


def test_attention_over_every_block_is_decode_attention():
    lens = [3000, 177]
    tables, nb = paged(lens, 1)
    kp, vp, q = (x.to(DEV) for x in (keys(nb, 2, 128, "bf16", 1), rand((nb, 2, 16, 128), torch.bfloat16, 2),
                                     rand((2, 8, 128), torch.bfloat16, 3)))
    sel = i32(np.broadcast_to(np.arange(188), (2, 2, 188)) * (np.arange(188) < np.array([188, 12])[:, None, None]) -
              (np.arange(188) >= np.array([188, 12])[:, None, None]))
    a = pkv.paged_decode_attention_sparse(q, kp, vp, i32(tables), i32(lens), sel, 0.05)
    b = pkv.paged_decode_attention(q, kp, vp, i32(tables), i32(lens), 0.05)
    pkv.paged_kv_check_status()
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -8 * b.float().abs().max()
