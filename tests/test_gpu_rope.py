"""GPU: rotary positions and the append that turns keys, against float64.

Bound of a turned value x cos a - y sin a against 64 bits: the fraction of a turn as
32 bits, then as a float32 in [-1, 1) (half a step, 2^-25, times pi) and sincospif
(2^-23) leave sine and cosine off by 2^-22 at most; two products and a sum round by
2^-24 of their size each: (|x| + |y|) factor 2^-20 holds them.  The frequency's 64-bit
form (a float64 product, 2^-52) moves an angle by 2^-51 of itself.  The output's own
rounding: eps/2 of it, or half the smallest subnormal."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, i32, rand
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def freqs(n, base=500000.0):
    return [base ** (-i / n) for i in range(n)]


def bound(x, pos, inv, dtype, interleaved, factor, ref):
    n = len(inv)
    a = np.abs(f64(x))
    i, j = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    mag = np.zeros_like(a)
    mag[..., i] = mag[..., j] = a[..., i] + a[..., j]
    far = np.abs(pos).max() * max(abs(f) for f in inv) * 2.0 ** -51
    u = torch.finfo(dtype).eps / 2
    tol = abs(factor) * mag * (2.0 ** -20 + far)
    return tol + np.where(mag > 0, u * (np.abs(ref) + tol) + torch.finfo(dtype).smallest_normal * u, 0.0)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 112)])
@pytest.mark.parametrize("tokens,hq,hk,axes,interleaved", [(1, 1, 1, 1, False), (1, 32, 8, 1, True), (3, 5, 5, 2, True),
                                                           (67, 7, 1, 3, False), (700, 6, 2, 4, True), (1301, 3, 2, 2, False),
                                                           (5000, 8, 2, 1, False)])
def test_rows(dtype, d, rot, tokens, hq, hk, axes, interleaved):
    dt = DT[dtype]
    q, k = rand((tokens, hq, d), dt, 1), rand((tokens, hk, d), dt, 2)
    rng = np.random.default_rng(tokens + rot)
    pos = rng.integers(0, 1 << 20, (axes, tokens))
    pos[0, 0] = 0
    axis = rng.integers(0, axes, rot // 2)
    axis[0] = axes - 1
    inv, factor = freqs(rot // 2), 1.0 if axes == 1 else 0.83
    rope = pkv.make_rope(inv, d, axes=axis, interleaved=interleaved, factor=factor)
    assert rope.num_axes == axes and rope.rot_dim == rot
    qo, ko = pkv.paged_kv_rope(q.to(DEV), k.to(DEV), i32(pos if axes > 1 else pos[0]), rope)
    for x, out in ((q, qo), (k, ko)):
        ref = lc.rope(f64(x), pos, inv, axis, interleaved, factor)
        assert_within(f64(out), ref, bound(x, pos, inv, dt, interleaved, factor, ref))
        assert torch.equal(out.cpu()[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16))
    pkv.paged_kv_check_status()


def test_extreme_positions():
    """The largest and negative positions: the angle from whole numbers."""
    from fractions import Fraction
    inv = [1.0, 0.75, 1e-3, 3.0, 0.5, 1e-9, 6.5, 2.0]
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 2 ** 30 + 7, 123456789, 0])
    k = torch.zeros(len(pos), 1, 64, dtype=torch.float16)
    k[..., :8] = 1.0                                              # cosine and sine appear as they are
    rope = pkv.make_rope(inv, 64)
    out = f64(pkv.paged_kv_rope(None, k.to(DEV), i32(pos), rope)[1])
    for t, p in enumerate(pos):
        for f, w in enumerate(inv):
            turn = Fraction(int(p)) * Fraction(w) / (2 * pi)
            a = float(2 * pi * (turn - turn.__floor__()))
            tol = 2.0 ** -20 + abs(int(p)) * w * 2.0 ** -51 + 2.0 ** -11
            assert abs(out[t, 0, f] - np.cos(a)) < tol and abs(out[t, 0, 8 + f] - np.sin(a)) < tol, (p, w)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_strides_and_in_place(dtype, d):
    """Parts of one projection, heads interleaved with others, and outputs that are the inputs."""
    dt, T, hq, hk = DT[dtype], 37, 6, 2
    rope = pkv.make_rope(freqs(d // 2), d)
    pos = i32(np.arange(T) * 31)
    qkv = rand((T, (hq + 2 * hk) * d), dt, 5).to(DEV)
    q, k, v = (x.view(T, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], -1))
    want = pkv.paged_kv_rope(q.contiguous(), k.contiguous(), pos, rope)
    got = pkv.paged_kv_rope(q, k, pos, rope)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = torch.zeros(T, hq, 3, d, dtype=dt, device=DEV)
    wide[:, :, 1] = q
    into = torch.zeros(T, hk + 3, d, dtype=dt, device=DEV)
    qo, ko = pkv.paged_kv_rope(wide[:, :, 1], k, pos, rope, q_out=wide[:, :, 1], k_out=into[:, 2:2 + hk])
    assert torch.equal(wide[:, :, 1], want[0]) and not wide[:, :, 0].any() and not wide[:, :, 2].any()
    assert torch.equal(into[:, 2:2 + hk], want[1]) and not into[:, :2].any() and not into[:, 2 + hk:].any()
    before = v.clone()
    pkv.paged_kv_rope(q, k, pos, rope, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 41, 610, 1300, 3000])
@pytest.mark.parametrize("fp8", [False, True], ids=["16-bit", "e4m3"])
def test_append_is_rope_then_append(dtype, d, tokens, fp8):
    dt, hq, hk = DT[dtype], 4, 2
    nb = tokens // 16 + 3
    rope = pkv.make_rope(freqs(d // 4), d, interleaved=True)      # half of the dims turn
    q, k, v = (rand((tokens, h, d), dt, i).to(DEV) for i, h in enumerate((hq, hk, hk)))
    pos = i32(np.arange(tokens) + 77)
    slots = np.random.default_rng(1).permutation(nb * 16)[:tokens].astype(np.int32)
    if tokens > 2:
        slots[1] = -1
    s = i32(slots)
    if fp8:
        pools = [torch.randint(0, 127, (nb, hk, 16, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.tensor([0.013, 0.5], device=DEV), torch.tensor([2.0, 0.01], device=DEV)]
    else:
        pools, scales = [rand((nb, hk, 16, d), dt, 9 + i).to(DEV) for i in range(2)], []
    ref = [p.clone() for p in pools]
    qo = pkv.paged_kv_append_rope(q, k, v, pos, rope, s, *pools, *scales)
    q2, k2 = pkv.paged_kv_rope(q, k, pos, rope)
    (pkv.paged_kv_append_fp8 if fp8 else pkv.paged_kv_append)(k2, v, s, *ref, *scales)
    pkv.paged_kv_check_status()
    assert torch.equal(qo, q2)
    for a, b in zip(pools, ref):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    # without queries
    again = [p.clone() for p in ref]
    assert pkv.paged_kv_append_rope(None, k, v, pos, rope, s, *again, *scales) is None
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, ref))


def test_slots_outside_the_pool_are_flagged():
    rope = pkv.make_rope(freqs(32), 64)
    k = rand((3, 1, 64), torch.float16, 0).to(DEV)
    pools = [torch.zeros(2, 1, 16, 64, dtype=torch.float16, device=DEV) for _ in range(2)]
    pkv.paged_kv_append_rope(None, k, k, i32([1, 2, 3]), rope, i32([5, 32, 2 ** 31 - 1]), *pools)
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_kv_check_status()
    assert e.value.code == -6
    assert pools[0][0, 0, 5].any() and not pools[0][1].any()
    pkv.paged_kv_check_status()


def test_dims_of_one_element_have_any_stride():
    rope = pkv.make_rope(freqs(32), 64)
    x = rand((7, 3, 64), torch.float16, 0).to(DEV)
    want = pkv.paged_kv_rope(x, x[:, :1].contiguous(), i32(range(7)), rope)
    odd = torch.as_strided(x, (7, 1, 64), (192, 5, 1))
    got = pkv.paged_kv_rope(x, odd, i32(range(7)), rope)
    assert torch.equal(got[1], want[1])
    one = torch.as_strided(x, (1, 3, 64), (3, 64, 1))
    assert torch.equal(pkv.paged_kv_rope(one, one, i32([0]), rope)[0], x[:1])


def test_no_tokens_other_stream_and_capture():
    rope = pkv.make_rope(freqs(64), 128)
    empty = torch.empty(0, 2, 128, dtype=torch.float16, device=DEV)
    qo, ko = pkv.paged_kv_rope(empty, empty, i32([]), rope)
    assert qo.shape == empty.shape and ko.shape == empty.shape
    q, k, pos = rand((9, 4, 128), torch.bfloat16, 0).to(DEV), rand((9, 2, 128), torch.bfloat16, 1).to(DEV), i32(range(9))
    want = pkv.paged_kv_rope(q, k, pos, rope)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pkv.paged_kv_rope(q, k, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.empty_like(q), torch.empty_like(k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_kv_rope(q, k, pos, rope, *out)
    pos += 5
    g.replay()
    want = pkv.paged_kv_rope(q, k, pos, rope)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    pkv.paged_kv_check_status()
