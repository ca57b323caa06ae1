"""Arguments that the rotary, chunk and block-sparse calls refuse before any launch (CPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, PkvRope, PkvRopeStrides, lib

INVALID, UNSUPPORTED = -1, -2
P = 1 << 20          # an address that is never read: every call here is refused, or has nothing to do


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def dims(**kw):
    base = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=8, max_blocks_per_seq=4,
                dtype=0)
    return ctypes.byref(PkvDims(**{**base, **kw}))


def rope(n=32, **kw):
    r = PkvRope()
    assert lib().paged_kv_rope_init(ctypes.byref(r), (ctypes.c_double * n)(*[0.5] * n), n, None, 1, 0, 1.0) == 0
    for k, v in kw.items():
        setattr(r, k, v)
    return ctypes.byref(r)


def test_rope_init():
    r, one = PkvRope(), (ctypes.c_double * 64)(*[1.0] * 64)

    def init(freqs=one, n=8, axes=None, num_axes=1, factor=1.0, dst=ctypes.byref(r)):
        return lib().paged_kv_rope_init(dst, freqs, n, axes, num_axes, 0, factor)

    assert init() == 0 and r.rot_dim == 16 and r.turns[0] == round(2.0 ** 64 * 0.15915494309189535)
    for kw in (dict(n=0), dict(n=12), dict(n=72), dict(num_axes=0), dict(num_axes=5), dict(factor=float("nan")), dict(dst=None),
               dict(freqs=None), dict(freqs=(ctypes.c_double * 8)(*[float("inf")] * 8)),
               dict(axes=(ctypes.c_int32 * 8)(0, 0, 0, 1, 0, 0, 0, 0)), dict(axes=(ctypes.c_int32 * 8)(*[-1] * 8))):
        assert init(**kw) == INVALID, kw
    assert init(axes=(ctypes.c_int32 * 8)(0, 0, 0, 1, 0, 0, 0, 3), num_axes=4) == 0


def test_rope_call():
    def call(q=P, k=P, pos=P, n=3, r=None, qo=P, ko=P, st=None, d=None):
        return lib().paged_kv_rope(q, k, pos, n, r if r is not None else rope(), qo, ko, st, d or dims(), 0)

    for kw in (dict(q=0), dict(k=0), dict(pos=0), dict(qo=0), dict(ko=0), dict(n=-1), dict(q=P + 8), dict(ko=P + 2),
               dict(pos=P + 1), dict(r=ctypes.POINTER(PkvRope)()), dict(r=rope(rot_dim=72)), dict(r=rope(rot_dim=128)),
               dict(r=rope(rot_dim=24)), dict(r=rope(num_axes=0)), dict(d=dims(num_q_heads=-1)),
               dict(st=ctypes.byref(PkvRopeStrides(q_token=4))), dict(st=ctypes.byref(PkvRopeStrides(k_head=-64)))):
        assert call(**kw) == INVALID, kw
    bits = rope()
    bits._obj.axis_bits[0] = 2
    assert call(r=bits) == INVALID
    for kw in (dict(d=dims(head_dim=96)), dict(d=dims(dtype=2)), dict(d=dims(num_q_heads=9000))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=0) == 0


def test_append_rope_call():
    def call(q=P, k=P, v=P, pos=P, slots=P, n=3, qo=P, kc=P, vc=P, ks=0, vs=0, d=None):
        return lib().paged_kv_append_rope(q, k, v, pos, slots, n, rope(), qo, kc, vc, ks, vs, None, d or dims(), 0)

    for kw in (dict(k=0), dict(v=0), dict(slots=0), dict(kc=0), dict(vc=0), dict(ks=P), dict(vs=P), dict(kc=P + 8),
               dict(ks=P, vs=P, vc=P + 4), dict(slots=P + 2), dict(v=P + 8), dict(n=-1)):
        assert call(**kw) == INVALID, kw
    assert call(d=dims(block_size=32)) == UNSUPPORTED
    assert call(n=0) == 0


def test_chunk_call():
    def call(q=P, k=P, v=P, t=P, l=P, o=P, n=5, scale=1.0, out=P, ws=P, nws=1 << 40, d=None):
        return lib().paged_chunk_attention(q, k, v, t, l, o, n, scale, out, ws, nws, d or dims(), 0)

    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(t=0), dict(l=0), dict(o=0), dict(out=0), dict(ws=0), dict(nws=4096),
               dict(ws=P + 16), dict(q=P + 8), dict(out=P + 8), dict(o=P + 2), dict(l=P + 1), dict(n=-1),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(d=dims(num_q_heads=5)), dict(d=dims(num_blocks=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=dims(num_q_heads=18)), dict(d=dims(head_dim=80)), dict(d=dims(num_seqs=8193)), dict(d=dims(dtype=2)),
               dict(d=dims(max_blocks_per_seq=1 << 27)), dict(n=2 ** 31 - 1, d=dims(max_blocks_per_seq=(1 << 27) - 1, num_q_heads=40000,
                                                                                    num_kv_heads=40000, num_blocks=1))):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=0) == 0 and call(d=dims(num_seqs=0)) == 0
    assert lib().paged_chunk_workspace_bytes(dims(head_dim=80)) == 0


def test_sparse_calls():
    def bounds(k=P, t=P, l=P, o=0, n=0, b=P, s=P, d=None):
        return lib().paged_kv_update_bounds(k, t, l, o, n, b, s, d or dims(), 0)

    for kw in (dict(k=0), dict(t=0), dict(l=0), dict(b=0), dict(s=0), dict(b=P + 8), dict(s=P + 2), dict(n=-1, o=P), dict(o=P + 2, n=1)):
        assert bounds(**kw) == INVALID, kw
    assert bounds(d=dims(num_seqs=0)) == 0 and bounds(o=P, n=0) == 0

    def select(q=P, b=P, s=P, t=P, l=P, num=3, sink=1, recent=1, sel=P, ws=P, nws=1 << 40, d=None):
        return lib().paged_select_blocks(q, b, s, t, l, num, sink, recent, sel, ws, nws, d or dims(), 0)

    for kw in (dict(q=0), dict(b=0), dict(s=0), dict(t=0), dict(l=0), dict(sel=0),
               dict(ws=0, d=dims(max_blocks_per_seq=257)), dict(nws=10, d=dims(max_blocks_per_seq=257)),
               dict(ws=P + 64, d=dims(max_blocks_per_seq=257)), dict(ws=0, d=dims(num_seqs=305)),
               dict(num=0), dict(sink=-1), dict(recent=0), dict(sink=3), dict(sink=2 ** 31 - 1, recent=5), dict(q=P + 4), dict(b=P + 4)):
        assert select(**kw) == INVALID, kw
    for kw in (dict(d=dims(num_seqs=70000)), dict(d=dims(num_q_heads=20)), dict(d=dims(head_dim=32))):
        assert select(**kw) == UNSUPPORTED, kw
    assert select(d=dims(num_seqs=0)) == 0
    # few sequences with tables of up to 256 blocks need no workspace
    need = lib().paged_select_workspace_bytes
    assert need(dims(max_blocks_per_seq=256)) == 0 and need(dims(max_blocks_per_seq=257)) > 0
    assert need(dims(num_seqs=304, num_kv_heads=1, num_q_heads=1)) == 0 < need(dims(num_seqs=305, num_kv_heads=1, num_q_heads=1))

    def sparse(q=P, k=P, v=P, t=P, l=P, sel=P, num=3, scale=1.0, out=P, d=None):
        return lib().paged_decode_attention_sparse(q, k, v, t, l, sel, num, scale, out, d or dims(), 0)

    for kw in (dict(q=0), dict(k=0), dict(v=0), dict(t=0), dict(l=0), dict(sel=0), dict(out=0), dict(num=-1), dict(v=P + 8),
               dict(sel=P + 2), dict(scale=float("nan"))):
        assert sparse(**kw) == INVALID, kw
    assert sparse(d=dims(num_seqs=65536)) == UNSUPPORTED and sparse(d=dims(num_seqs=0)) == 0


def test_binding_refuses_before_the_library():
    f = torch.zeros(3, 2, 64, dtype=torch.float16)
    cache, i = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    r = pkv.make_rope([0.5] * 32, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_rope(f, f, i, r)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_append_rope(f, f, f, i, r, i, cache, cache)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_chunk_attention(f, cache, cache, i[:, None], i, torch.zeros(4, dtype=torch.int32), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_kv_update_bounds(cache, i[:, None], i, torch.zeros(4, 2, 2, 64, dtype=torch.int8), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_select_blocks(f, torch.zeros(4, 2, 2, 64, dtype=torch.int8), torch.zeros(4, 2), i[:, None], i, 3)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_decode_attention_sparse(f, cache, cache, i[:, None], i, torch.zeros(3, 2, 1, dtype=torch.int32), 1.0)
    for bad in (dict(inv_freq=[1.0] * 40, head_dim=64), dict(inv_freq=[1.0] * 8, head_dim=64, axes=[0] * 7)):
        with pytest.raises(ValueError):
            pkv.make_rope(**bad)
    for bad in (dict(inv_freq=[1.0] * 7, head_dim=64), dict(inv_freq=[float("nan")] * 8, head_dim=64),
                dict(inv_freq=[1.0] * 8, head_dim=64, axes=[4] * 8)):
        with pytest.raises(pkv.PagedKVError):
            pkv.make_rope(**bad)
