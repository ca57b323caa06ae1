"""GPU block tables and draft verification, the parts that need no GPU: the
oracle against the host allocator's own rules and against the target's
distribution, and the entry points' refusals."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from oracle import serving
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvVerifyDims, lib


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def test_resize_slots_are_the_host_mapping_of_the_new_tokens():
    rng = np.random.default_rng(0)
    for _ in range(20):
        B, MB, nb = 6, 9, 60
        lens = rng.integers(0, 100, B)
        grow = rng.integers(0, 6, B)
        tables = np.full((B, MB), -1, np.int32)
        perm = list(rng.permutation(nb))
        for b in range(B):
            for j in range(-(-lens[b] // 16)):
                tables[b, j] = perm.pop()
        free = np.array(perm + [-1] * (nb - len(perm)))
        slots, offs, after, lst, cnt = serving.resize_tables(lens, lens + grow, tables, free, len(perm))
        for b in range(B):
            for i in range(grow[b]):  # the newest token's slot of every length on the way
                n = np.array([lens[b] + i + 1], np.int32)
                assert slots[offs[b] + i] == pkv.paged_kv_slot_mapping(after[b:b + 1], n)[0]
        held = [int(after[b, j]) for b in range(B) for j in range(-(-(lens[b] + grow[b]) // 16))]
        assert sorted(held + lst[:cnt]) == list(range(nb))
        # taken back, the list is as it was
        _, _, _, lst2, cnt2 = serving.resize_tables(lens + grow, lens, after, lst, cnt)
        assert cnt2 == len(perm) and lst2[:cnt2] == perm


def test_resize_example():
    tables = np.array([[5, -1, -1], [7, 3, -1], [-1, -1, -1]], np.int32)
    # sequence 0 grows over a border, 1 gives a block back, 2 starts
    slots, offs, t, free, n = serving.resize_tables([16, 20, 0], [18, 16, 1], tables, [9, 8, -1, -1], 2)
    assert slots == [3 * 16, 3 * 16 + 1, 8 * 16] and offs == [0, 2, 2, 3]  # the given block is on top
    assert t[0, 1] == 3 and t[2, 0] == 8 and n == 1 and free[:1] == [9]
    assert serving.resize_tables([0], [33], tables[:1], [1, 2], 2) is None


def test_weights_and_draws():
    assert serving.weight(1.0) == 1 << 40 and serving.weight(2.0) == 1 << 40
    assert serving.weight(-1.0) == serving.weight(float("nan")) == serving.weight(0.0) == 0
    assert serving.weight(2.0 ** -41) == 0 and serving.weight(3 * 2.0 ** -41) == 2  # ties to even
    assert serving.draw([0, 4, 0, 4], 0.0) == 1 and serving.draw([0, 4, 0, 4], 0.5) == 3
    assert serving.draw([0, 4, 0, 4], 1.0) == 3 and serving.draw([0, 0], 0.3) == -1
    assert serving.draw([0, 4, 0, 4], float("nan")) == 1


def test_verification_has_the_targets_distribution():
    """Over all drafts, acceptances and draws, token v comes out with probability p(v)."""
    p = [Fraction(x, 64) for x in (20, 0, 10, 30, 4)]
    q = [Fraction(x, 64) for x in (10, 14, 20, 20, 0)]
    out = [Fraction(0)] * 5
    for x in range(5):
        if q[x] == 0:
            continue
        keep = min(Fraction(1), p[x] / q[x])
        # the oracle accepts exactly the u below p/q
        eps = 2.0 ** -20
        if 0 < keep < 1:
            for u, want in ((float(keep) - eps, 1), (float(keep) + eps, 0)):
                a, _ = serving.verify_one([list(map(float, p))] * 2, [list(map(float, q))], [x], 1, [u], 0.0)
                assert a == want
        out[x] += q[x] * keep
        rest = [max(serving.weight(float(a)) - serving.weight(float(b)), 0) for a, b in zip(p, q)]
        for v in range(5):
            out[v] += q[x] * (1 - keep) * Fraction(rest[v], sum(rest))
    assert out == p


def test_c_refusals():
    p, odd, null = ctypes.c_void_p(4096), ctypes.c_void_p(4098), ctypes.c_void_p(0)

    def resize(cl=p, nl=p, B=2, MB=3, bs=16, bt=p, fb=p, nf=p, nb=8, sm=p, ns=4, to=p):
        return lib().paged_kv_resize_tables(cl, nl, B, MB, bs, bt, fb, nf, nb, sm, ns, to, null)

    assert resize(B=-1) == resize(MB=-1) == resize(nb=0) == resize(ns=-1) == -1
    assert resize(cl=null) == resize(nl=null) == resize(bt=null) == resize(fb=null) == resize(nf=null) == -1
    assert resize(sm=null) == -1 and resize(cl=odd) == resize(to=odd) == -1
    assert resize(bs=32) == resize(B=8193) == resize(nb=1 << 27) == resize(MB=1 << 27) == -2
    assert resize(B=8192, MB=1 << 18) == -2

    def verify(t=p, d=p, x=p, dl=p, au=p, su=p, cl=p, na=p, ot=p, nl=p, B=1, K=2, V=10, dt=2, s=(30, 10, 20, 10)):
        dims = PkvVerifyDims(B, K, V, dt, *s)
        return lib().paged_verify_draft(t, d, x, dl, au, su, cl, ctypes.byref(dims), na, ot, nl, null)

    assert verify(B=0) == 0
    assert verify(B=-1) == verify(K=-1) == verify(V=0) == -1
    assert verify(dt=3) == verify(K=32) == verify(V=(1 << 22) + 1) == -2
    assert verify(t=null) == verify(x=null) == verify(au=null) == verify(su=null) == verify(na=null) == -1
    assert verify(ot=null) == verify(cl=null) == -1          # new_lens needs context_lens
    assert verify(t=odd) == verify(s=(-1, 1, 1, 1)) == -1
    assert lib().paged_verify_draft(p, p, p, p, p, p, p, None, p, p, p, null) == -1


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.paged_kv_resize_tables(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1])
    with pytest.raises(ValueError):
        pkv.paged_verify_draft(torch.zeros(2, 2, 5), None, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1),
                               torch.zeros(2))
