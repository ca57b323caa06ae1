"""The 4-bit format on the CPU: the oracle against closed forms and the
contract's own bounds, the binding's refusals before any launch, and the C
entry points' refusals (which need no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from oracle import int4
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, lib


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_byte_order_is_a_bijection(d, is_v):
    at, shift = int4.code_map(d, is_v)
    nibbles = (2 * at + shift // 4).flatten()
    assert sorted(nibbles) == list(range(16 * d))


def test_closed_forms():
    # a ramp of 16 levels is held without loss; so is a constant row
    x = np.tile(np.arange(16, dtype=np.float32) * 0.25 - 2.0, 4)[None]
    codes, pairs = int4.quantise_rows(x)
    assert np.array_equal(codes[0], np.tile(np.arange(16), 4))
    assert list(pairs[0]) == [np.float16(0.25), np.float16(-2.0)]
    codes, pairs = int4.quantise_rows(np.full((1, 64), 3.5, np.float32))
    assert not codes.any() and list(pairs[0]) == [0, np.float16(3.5)]
    # values past the float16 range are limited to it
    codes, pairs = int4.quantise_rows(np.array([[np.inf, -np.inf] * 32], np.float32))
    assert list(pairs[0].astype(np.float64)) == [float(np.float16(131008 / 15)), -65504.0]
    assert set(codes[0]) == {0, 15}


@pytest.mark.parametrize("d", [64, 128])
def test_append_then_values_is_within_half_a_step(d):
    rng = np.random.default_rng(d)
    hk, nb, n = 3, 4, 23
    rows = (rng.standard_normal((n, hk, d)) * np.exp(rng.uniform(-6, 6, (n, hk, 1)))).astype(np.float16)
    slots = rng.permutation(nb * 16)[:n].astype(np.int32)
    slots[5] = -1
    for is_v in (False, True):
        pool = np.full((nb, hk, 16, d // 2 + 4), 0xFF, np.uint8)
        out = int4.append_one(pool, rows.astype(np.float32), slots, is_v)
        v = int4.values(out, is_v).transpose(0, 2, 1, 3).reshape(nb * 16, hk, d)
        _, pairs = int4.quantise_rows(rows)
        for i, s in enumerate(slots):
            if s < 0:
                continue
            x, sc = rows[i].astype(np.float64), pairs[i, :, :1].astype(np.float64)
            # half a step; the scale itself is rounded to float16 (2^-11 of 15 steps, and 2^-25 where it is subnormal)
            bound = sc * 0.5 + 15 * (sc * 2.0 ** -11 + 2.0 ** -25) + 2.0 ** -22 * np.abs(x).max()
            assert np.all(np.abs(v[s] - x) <= bound)
        touched = np.zeros(nb * 16, bool)
        touched[slots[slots >= 0]] = True
        assert np.isnan(v[~touched]).all()  # the other rows kept their bytes


def test_append_leaves_the_neighbours_bytes():
    rng = np.random.default_rng(0)
    pool = rng.integers(0, 256, (2, 2, 16, 68)).astype(np.uint8)
    rows = rng.standard_normal((1, 2, 128)).astype(np.float32)
    for is_v in (False, True):
        out = int4.append_one(pool, rows, np.array([19]), is_v)
        at, _ = int4.code_map(128, is_v)
        mine = np.zeros(16 * 68, bool)
        mine[at[3]] = True
        mine[8 * 128 + 12:8 * 128 + 16] = True
        a, b = int4.tiles(pool), int4.tiles(out)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1][:, ~mine], b[1][:, ~mine])


def test_attention_of_the_oracle_is_attention_over_the_values():
    rng = np.random.default_rng(1)
    pool = np.full((2, 5, 1, 16, 36), 0, np.uint8)
    rows = rng.standard_normal((2, 37, 1, 64)).astype(np.float32)
    tables = np.array([[4, 0, 2]], np.int32)
    slots = np.array([tables[0, p // 16] * 16 + p % 16 for p in range(37)])
    k = int4.append_one(pool[0], rows[0], slots, False)
    v = int4.append_one(pool[1], rows[1], slots, True)
    q = rng.standard_normal((1, 2, 64))
    out = int4.decode_attention(q, k, v, tables, [37], 0.125)
    kk, vv = (int4.values(p, f).transpose(0, 2, 1, 3).reshape(-1, 64)[slots] for p, f in ((k, False), (v, True)))
    ref = torch.softmax(torch.from_numpy(q[0]) @ torch.from_numpy(kk).T * 0.125, -1) @ torch.from_numpy(vv)
    assert np.allclose(out[0], ref.numpy(), rtol=0, atol=1e-12)


def _dims(**kw):
    d = dict(num_seqs=2, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_blocks=4,
             max_blocks_per_seq=2, dtype=1)
    d.update(kw)
    return PkvDims(**d)


def test_c_refusals():
    p = ctypes.c_void_p(4096)
    odd = ctypes.c_void_p(4104)
    null = ctypes.c_void_p(0)

    def append(k=p, v=p, s=p, n=1, kc=p, vc=p, **kw):
        return lib().paged_kv_append_int4(k, v, s, n, kc, vc, ctypes.byref(_dims(**kw)), null)

    def read(s=p, n=1, kc=p, vc=p, k=p, v=p, **kw):
        return lib().paged_kv_read_int4(s, n, kc, vc, k, v, ctypes.byref(_dims(**kw)), null)

    def attend(q=p, kc=p, vc=p, bt=p, cl=p, scale=0.1, out=p, ws=p, n=0, **kw):
        return lib().paged_decode_attention_int4(q, kc, vc, bt, cl, scale, out, ws, n, ctypes.byref(_dims(**kw)), null)

    for f in (append, read):
        assert f(n=0) == 0                          # nothing to do
        assert f(n=-1) == -1
        assert f(k=null) == f(kc=null) == f(s=null) == -1
        assert f(k=odd) == f(vc=odd) == -1          # 16-byte alignment
        assert f(head_dim=80) == f(block_size=32) == f(dtype=2) == -2
        assert f(num_blocks=0) == -1
        assert f(num_blocks=1 << 30) == -2          # rows past 2^31
    assert attend(num_seqs=0) == 0
    assert attend(num_seqs=2049) == -2
    assert attend(num_q_heads=7) == -1 and attend(num_q_heads=18) == -2
    assert attend(q=null) == attend(bt=null) == attend(out=odd) == -1
    assert attend(scale=float("nan")) == -1
    assert attend(n=64) == -1                       # workspace too small
    assert lib().paged_decode_step_int4(p, null, p, p, p, p, p, 0.1, p, p, 0, ctypes.byref(_dims()), null) == -1
    assert lib().paged_kv_append_int4(p, p, p, 1, p, p, None, null) == -1


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, 68, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pkv.paged_kv_append_int4(k, k, torch.zeros(4, dtype=torch.int32), pool, pool)
    with pytest.raises(ValueError):
        pkv.paged_kv_read_int4(torch.zeros(4, dtype=torch.int32), pool, pool, torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_int4(torch.zeros(1, 2, 128, dtype=torch.bfloat16), pool, pool,
                                        torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 0.1)
