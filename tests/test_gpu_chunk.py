"""GPU: attention of chunks of new tokens against float64 (the bound is derived in
long_context_helpers.tolerance)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, hide_tails, i32, paged, rand, tolerance
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def inputs(new, lens, hq, hk, d, dtype, seed=0, extra=3, spread=1.0):
    """q, pools with NaN where no token is, tables, offsets (CPU)."""
    tables, nb = paged(lens, seed, extra)
    dt = DT[dtype]
    pools = [hide_tails(rand((nb, hk, 16, d), dt, seed + i), tables, lens) for i in (1, 2)]
    q = rand((int(sum(new)), hq, d), dt, seed + 3, spread)
    return q, pools[0], pools[1], tables, np.concatenate([[0], np.cumsum(new)])


def run(q, kp, vp, tables, lens, offsets, scale, **kw):
    out = pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32(lens), i32(offsets), scale, **kw)
    pkv.paged_kv_check_status()
    return out


def check(out, q, kp, vp, tables, lens, offsets, scale, what=""):
    ref, mag = lc.chunk_attention(f64(q), f64(kp), f64(vp), tables, lens, offsets, scale)
    r = slice(int(offsets[0]), int(offsets[-1]))
    k, v = f64(kp), f64(vp)
    tol = tolerance(ref[r], mag[r], q.dtype, f64(q)[r], k, v, scale, max([1, *map(int, lens)]))
    assert_within(f64(out)[r], ref[r], tol, what)


# new tokens and contexts: one token; a whole prompt; a mix with empty slots; tiles that end at, before and after 16,
# 128 and 256; chunks of long contexts
RAGGED = [([1], [1]), ([1], [300]), ([5], [5]), ([17], [33]), ([128], [128]), ([129], [257]), ([64, 1, 0, 40], [64, 130, 50, 41]),
          ([0, 3, 0], [0, 3, 9]), ([300], [300]), ([33, 127, 1], [1000, 127, 513]), ([7], [2050])]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (3, 1), (8, 2), (5, 1), (6, 1), (14, 2), (8, 1)])
def test_ragged(dtype, d, hq, hk):
    for i, (new, lens) in enumerate(RAGGED):
        a = inputs(new, lens, hq, hk, d, dtype, seed=i)
        out = run(*a[:4], lens, a[4], d ** -0.5)
        check(out, *a[:4], lens, a[4], d ** -0.5, (new, lens))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hq,hk,new,lens", [
    (128, 8, 2, [700], [700]),                      # several units a head, all cut differently
    (64, 4, 4, [1500, 2], [1500, 700]),
    (128, 4, 1, [16], [20000]),                     # one unit over many CTAs
    (64, 8, 1, [1], [9000]),
    (128, 2, 2, [513, 257, 1, 1, 1], [1025, 300, 4097, 1, 128])])
def test_cut_units(dtype, d, hq, hk, new, lens):
    a = inputs(new, lens, hq, hk, d, dtype, seed=11)
    out = run(*a[:4], lens, a[4], d ** -0.5)
    check(out, *a[:4], lens, a[4], d ** -0.5)


# (new tokens, contexts) on both sides of the longest context whose units are never cut, and of as many units as CTAs
@pytest.mark.parametrize("new,lens", [([1, 3, 0, 200], [1024, 1000, 9, 200]), ([1, 3], [1025, 70]), ([1024], [1024]),
                                      ([600, 1], [1025, 1]), ([1] * 75, [1000] * 74 + [1024]), ([1] * 77, [900] * 77),
                                      ([1] * 200, list(range(1, 201)))])
@pytest.mark.parametrize("width", [0, 64, 65, 300])
def test_units_that_are_not_cut(new, lens, width):
    """Short contexts in tables that end with them and in wide ones."""
    d, dtype = (64, "bf16") if width % 2 else (128, "fp16")
    q, kp, vp, tables, off = inputs(new, lens, 6, 2, d, dtype, seed=width)
    wide = np.full((len(lens), max(width, tables.shape[1])), -1, np.int32)
    wide[:, :tables.shape[1]] = tables
    check(run(q, kp, vp, wide, lens, off, d ** -0.5), q, kp, vp, wide, lens, off, d ** -0.5, (new, lens, width))


def test_many_sequences():
    rng = np.random.default_rng(5)
    new = rng.integers(0, 6, 900)
    lens = new + rng.integers(0, 60, 900)
    a = inputs(new, lens, 4, 2, 64, "bf16", seed=3)
    out = run(*a[:4], lens, a[4], 0.125)
    check(out, *a[:4], lens, a[4], 0.125)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3e-6, 1.7])
@pytest.mark.parametrize("far", [[], [2500]])       # with a long context units are cut
def test_scales(dtype, scale, far):
    new, lens = [30, 200] + [2] * len(far), [150, 200] + far
    a = inputs(new, lens, 4, 2, 128, dtype, seed=7, spread=0.5)
    out = run(*a[:4], lens, a[4], scale)
    check(out, *a[:4], lens, a[4], scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_references_that_move(dtype, d):
    """Logits that rise from tile to tile by far more than 2^8, fall, and rise again."""
    lens, new = [1200], [40]
    q, kp, vp, tables, off = inputs(new, lens, 4, 2, d, dtype, seed=2)
    pos = np.arange(1200)
    gain = np.where(pos < 700, pos / 100, np.where(pos < 900, 0.1, 12.0))
    for j in range(75):
        kp[tables[0, j]] = (kp[tables[0, j]].float() * torch.from_numpy(gain[16 * j:16 * j + 16, None]).float()).to(kp.dtype)
    out = run(q, kp, vp, tables, lens, off, 0.5)
    check(out, q, kp, vp, tables, lens, off, 0.5)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("far", [[], [3000]])       # with a long context units are cut
def test_values_that_are_not_finite(dtype, d, hq, hk, far):
    """NaN and infinities of later tokens do not reach earlier rows; of visible ones they do."""
    new, lens = [150, 20] + [1] * len(far), [230, 20] + far
    q, kp, vp, tables, off = inputs(new, lens, hq, hk, d, dtype, seed=4)

    def put(pool, b, pos, h, dim, value):
        pool[tables[b, pos // 16], h, pos % 16, dim] = value

    put(vp, 0, 100, 0, 3, float("inf"))             # seen by rows 20 .. of sequence 0
    put(vp, 0, 170, 0, 3, float("-inf"))            # with the other: NaN from row 90
    put(vp, 0, 229, hk - 1, d - 1, float("nan"))    # the last row alone
    put(vp, 1, 7, 0, 0, float("-inf"))
    put(kp, 1, 12, 0, 5, float("nan"))              # a key: all of the rows that see it
    out = run(q, kp, vp, tables, lens, off, 0.3)
    ref, mag = lc.chunk_attention(f64(q), f64(kp), f64(vp), tables, lens, off, 0.3)
    got = f64(out)
    g = hq // hk
    assert np.isnan(got[150 + 12:170, :g]).all() and np.isnan(ref[150 + 12:170, :g]).all()
    tol = tolerance(np.nan_to_num(ref, posinf=0, neginf=0), mag, q.dtype, f64(q), f64(kp), f64(vp), 0.3, max(lens))
    keep = np.ones_like(ref, bool)
    keep[150 + 12:170, :g] = False
    if dtype == "fp16":
        # A weight below 2^-25 beside a largest one of 1 rounds to 0 in fp16, and 0 times infinity is NaN:
        # 64 bits keep the weight and give the infinity.
        keep &= ~(np.isinf(ref) & np.isnan(got))
    assert_within(np.where(keep, got, 0), np.where(keep, ref, 0), tol)
    assert not np.isfinite(got[20:90, 0, 3]).any() and np.isfinite(got[:20]).all() and np.isfinite(got[149, 0, 4])


def test_rows_outside_the_offsets_keep_what_they_hold():
    new, lens = [3, 5], [9, 5]
    q, kp, vp, tables, off = inputs([2, *new, 4], [2, *lens, 4], 4, 2, 64, "fp16", seed=1)
    tables, off = tables[1:3], np.array([2, 5, 10])
    out = torch.full((q.shape[0], 4, 64), 7.5, dtype=q.dtype, device=DEV)
    got = run(q, kp, vp, tables, lens, off, 0.125, out=out)
    assert got is out and (out[:2] == 7.5).all() and (out[10:] == 7.5).all()
    check(out, q, kp, vp, tables, lens, off, 0.125)


def test_contexts_shorter_than_the_chunk():
    for new, lens in (([40], [13]), ([300], [20]), ([5], [0]), ([600, 4], [170, 4])):
        a = inputs(new, lens, 8, 2, 128, "bf16", seed=6)
        out = run(*a[:4], lens, a[4], 0.1)
        check(out, *a[:4], lens, a[4], 0.1)
        assert not out[:new[0] - lens[0]].any()


def test_shared_blocks_and_small_pool_type():
    """Two sequences over the same prefix, in a pool without spare blocks."""
    lens, new = [100, 90], [4, 26]
    tables, nb = paged([100], 0, 3, width=7)
    tables = np.concatenate([tables, tables])
    tables[1, 4:6] = [i for i in range(nb) if i not in tables[0]][:2]
    pools = [rand((nb, 2, 16, 64), torch.float16, i) for i in (1, 2)]
    q = rand((30, 4, 64), torch.float16, 3)
    off = np.array([0, 4, 30])
    check(run(q, *pools, tables, lens, off, 0.2), q, *pools, tables, lens, off, 0.2)


def test_bad_tables_lengths_and_offsets_are_flagged():
    q, kp, vp, tables, off = inputs([4, 8], [40, 8], 4, 2, 64, "fp16")

    def flagged(t, l, o):
        out = pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(t), i32(l), i32(o), 0.125)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == -6
        pkv.paged_kv_check_status()
        return out

    bad = tables.copy()
    bad[0, 1] = kp.shape[0]                          # reads as zeros
    got = flagged(bad, [40, 8], off)
    zk, zv = torch.cat([kp, torch.zeros_like(kp[:1])]), torch.cat([vp, torch.zeros_like(vp[:1])])
    check(got, q, zk, zv, bad, [40, 8], off, 0.125)
    flagged(tables, [1000, 8], off)                  # longer than its table: limited
    flagged(tables, [40, -1], off)
    flagged(tables, [40, 8], [0, 13, 12])            # past the rows, and falling
    flagged(tables, [40, 8], [-1, 4, 12])
    flagged(tables, [40, 8], [0, 9, 4])


def test_workspace_streams_and_capture():
    new, lens = [3, 40], [2000, 300]
    q, kp, vp, tables, off = inputs(new, lens, 8, 2, 128, "bf16", seed=9)
    dev = [x.to(DEV) for x in (q, kp, vp)] + [i32(tables), i32(lens), i32(off)]
    ws = pkv.make_workspace_chunk(dev[0], dev[1], dev[3])
    ws.fill_(255)
    want = pkv.paged_chunk_attention(*dev, 0.1, workspace=ws)
    check(want, q, kp, vp, tables, lens, off, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pkv.paged_chunk_attention(*dev, 0.1, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # captured once, replayed with other lengths and offsets written on the stream
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_chunk_attention(*dev, 0.1, out=out, workspace=ws)
    dev[4].copy_(i32([1500, 40]))
    dev[5].copy_(i32([0, 5, 43]))
    for _ in range(3):
        g.replay()
    check(out, q, kp, vp, tables, [1500, 40], [0, 5, 43], 0.1)
    pkv.paged_kv_check_status()
    # the same call again gives the same bits; a second heads layout shares the workspace
    again = pkv.paged_chunk_attention(*dev, 0.1, workspace=ws)
    assert torch.equal(again, out)


def test_after_other_kernels_of_the_stream():
    """Lengths, offsets and the cache written right before the call."""
    new, lens = [5, 30], [400, 30]
    q, kp, vp, tables, off = inputs(new, lens, 4, 2, 64, "fp16", seed=10)
    dev = [x.to(DEV) for x in (q, kp, vp)] + [i32(tables)]
    blank = [torch.zeros_like(x) for x in dev[1:3]]
    l, o = i32([1, 1]), i32([0, 1, 2])
    real_l, real_o = i32(lens), i32(off)
    big = torch.empty(1 << 26, device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        big.fill_(1.0)
        blank[0].copy_(dev[1])
        blank[1].copy_(dev[2])
        l.copy_(real_l)
        o.copy_(real_o)
        out = pkv.paged_chunk_attention(dev[0], *blank, dev[3], l, o, 0.125)
    check(out, q, kp, vp, tables, lens, off, 0.125)


def test_no_tokens():
    q, kp, vp, tables, _ = inputs([2], [2], 2, 1, 64, "fp16")
    out = pkv.paged_chunk_attention(q[:0].to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32([2]), i32([0, 0]), 1.0)
    assert out.shape == (0, 2, 64)
    out = torch.full((2, 2, 64), 3.0, dtype=torch.float16, device=DEV)
    pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32([2]), i32([0, 0]), 1.0, out=out)
    pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables[:0]), i32([]), i32([0]), 1.0, out=out)
    assert (out == 3.0).all()
    pkv.paged_kv_check_status()


def test_pool_past_4_gb():
    """Blocks whose bytes lie past 2^32."""
    hk, d = 8, 128
    nb = (5 << 30) // (hk * 16 * d * 2)
    kp = torch.zeros(nb, hk, 16, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    lens, new = [130], [9]
    ids = np.concatenate([[nb - 1, 0, nb - 2], nb // 2 + np.arange(6)]).astype(np.int32)
    small = [rand((9, hk, 16, d), torch.bfloat16, i) for i in (1, 2)]
    for p, s in zip((kp, vp), small):
        p[torch.from_numpy(ids.astype(np.int64)).to(DEV)] = s.to(DEV)
    q = rand((9, 32, d), torch.bfloat16, 3)
    out = pkv.paged_chunk_attention(q.to(DEV), kp, vp, i32(ids[None]), i32(lens), i32([0, 9]), 0.09)
    pkv.paged_kv_check_status()
    check(out, q, *small, np.arange(9)[None], lens, np.array([0, 9]), 0.09)
