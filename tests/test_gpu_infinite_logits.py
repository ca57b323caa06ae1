"""GPU: logits of -infinity.  A key that holds one has weight 0 beside finite logits, and a
row whose visible logits are all -infinity is NaN, as softmax is; a row that sees no key
stays zero.  (Bounds: long_context_helpers.tolerance.)"""
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


def inputs(rows, lens, hq, hk, d, dtype, lost, seed=0):
    """Queries whose dim 2 is positive, and pools whose keys at positions lost[b] of KV head 0 hold -infinity there."""
    tables, nb = paged(lens, seed)
    kp, vp = (hide_tails(rand((nb, hk, 16, d), DT[dtype], seed + i), tables, lens) for i in (1, 2))
    for b, positions in enumerate(lost):
        for p in positions:
            kp[tables[b, p // 16], 0, p % 16, 2] = float("-inf")
    q = rand((rows, hq, d), DT[dtype], seed + 3)
    q[..., 2] = q[..., 2].abs() + 0.25
    return q, kp, vp, tables


# new tokens, lengths, positions of -infinity; the long contexts are cut between CTAs
CHUNKS = [([5, 9], [5, 9], [range(3), [4]]),                            # rows 0 .. 2 see nothing else
          ([200], [200], [range(130)]),                                 # more than a tile of them
          ([40, 3], [3000, 700], [range(2970), range(700)]),            # the pieces of all CTAs but the last
          ([30], [2500], [list(range(1400)) + list(range(2480, 2500))]),
          ([20, 300], [13, 120], [range(6), range(120)])]               # beside rows without any key


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1), (128, 3, 3)])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
@pytest.mark.parametrize("sign", [1, -1])
def test_chunk(dtype, d, hq, hk, case, sign):
    new, lens, lost = CHUNKS[case]
    q, kp, vp, tables = inputs(sum(new), lens, hq, hk, d, dtype, lost, seed=case)
    kp, scale, off = sign * kp, sign * 0.2, np.concatenate([[0], np.cumsum(new)])
    out = pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32(lens), i32(off), scale)
    pkv.paged_kv_check_status()
    ref, mag = lc.chunk_attention(f64(q), f64(kp), f64(vp), tables, lens, off, scale)
    g = hq // hk
    for b, (n, length) in enumerate(zip(new, lens)):
        for i in range(n):
            seen = range(max(length - n + i + 1, 0))
            empty = len(seen) > 0 and set(seen) <= set(lost[b])
            row = ref[off[b] + i]
            assert np.isnan(row[:g]).all() if empty else np.isfinite(row[:g]).all() and (len(seen) > 0 or not row.any())
            assert np.isfinite(row[g:]).all()
    assert_within(f64(out), ref, tolerance(ref, mag, DT[dtype], f64(q), f64(kp), f64(vp), scale, max(lens)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
@pytest.mark.parametrize("num", [3, 300])           # one CTA; a cluster of them
def test_sparse(dtype, d, hq, hk, num):
    """Blocks of nothing but -infinity, a last one of one token among them, alone and beside others."""
    lens = [33, 33, 16, 4801, 4801, 0]
    lost = [[32], range(33), range(16), list(range(16, 4000)) + [4800], range(4801), []]
    q, kp, vp, tables = inputs(len(lens), lens, hq, hk, d, dtype, lost)
    sel = np.full((len(lens), hk, num), -1, np.int32)
    rng = np.random.default_rng(num)
    for b, n in enumerate(lens):
        some = rng.permutation(-(-n // 16))[:num]
        sel[b, :, :len(some)] = some
    sel[3, :, :3] = [300, 5, 0]
    out = pkv.paged_decode_attention_sparse(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32(lens), i32(sel), 0.2)
    pkv.paged_kv_check_status()
    ref, mag = lc.sparse_attention(f64(q), f64(kp), f64(vp), tables, lens, sel, 0.2)
    g = hq // hk
    for b, nan in enumerate([False, True, True, False, True, False]):
        assert np.isnan(ref[b, :g]).all() == nan and np.isfinite(ref[b, g:]).all()
    assert not ref[5].any()
    bits = 11 if dtype == "fp16" else 16
    assert_within(f64(out), ref, tolerance(ref, mag, DT[dtype], f64(q), f64(kp), f64(vp), 0.2, 16 * num, bits))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("length", [900, 3000])     # whole; cut between CTAs
def test_infinite_values_at_weights_of_zero(dtype, length):
    """0 times infinity is NaN, in the piece of a unit that holds no weight as well."""
    q, kp, vp, tables = inputs(40, [length], 4, 2, 128, dtype, [range(800)])
    vp[tables[0, 0], 0, 5, 3] = float("inf")
    vp[tables[0, 40], 0, 7, 6] = float("nan")
    off, sel = np.array([0, 40]), np.arange(-(-length // 16), dtype=np.int32)[None, None].repeat(2, 1)
    chunk = pkv.paged_chunk_attention(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32([length]), i32(off), 0.2)
    sparse = pkv.paged_decode_attention_sparse(q[:1].to(DEV), kp.to(DEV), vp.to(DEV), i32(tables), i32([length]), i32(sel), 0.2)
    pkv.paged_kv_check_status()
    for got, (ref, mag), x, bits in (
            (chunk, lc.chunk_attention(f64(q), f64(kp), f64(vp), tables, [length], off, 0.2), q, None),
            (sparse, lc.sparse_attention(f64(q[:1]), f64(kp), f64(vp), tables, [length], sel, 0.2), q[:1], 11 if dtype == "fp16" else 16)):
        assert np.isnan(ref[:, :2, [3, 6]]).all() and np.isnan(ref).sum() == ref.shape[0] * 4
        assert_within(f64(got), ref, tolerance(np.nan_to_num(ref), mag, DT[dtype], f64(x), f64(kp), f64(vp), 0.2, length, bits))
