"""4-bit attention where V rows of one context differ widely in scale, and rows
that hold a NaN.

The bound of test_gpu_int4 takes the largest row attended; here every row
counts by its softmax weight p_t, so that a row without weight may not cost the
others anything:
  |gpu - ref| <= (2^-11 + n 2^-25) H + 2^-13 A + n 2^-46 + u |ref| + w
with H = sum p_t 7.5 s_t (each product p_t s_t is rounded to float16, 2^-11 of
it, and multiplies c - 7.5 steps; a product in float16's subnormal range is off
by 2^-25 instead, in units in which the largest product of the piece is at least
1, so that n of them move the mean by at most n 2^-25 of H, or, where the largest
belongs to a row of scale 0, which counts as 2^-24, by n 7.5 2^-25 / 2^24),
A = sum p_t max|V_t| (the weights' own errors, relative to each weight, as in
test_gpu_int4: 2^-14, in numerator and normaliser), u and w the output's
rounding as there."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from oracle import int4
from paged_kv_cache_26_gb300 import build as pkv_build
from parity_helpers import bits, widen_out

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.float16: "fp16", torch.bfloat16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def pools_of(k, v, table, nb):
    """4-bit pools (numpy) holding rows k / v [n][Hkv][D] at a table's positions; other slots 0xFF."""
    n, hk, d = k.shape
    slots = table[np.arange(n) // 16] * 16 + np.arange(n) % 16
    empty = np.full((nb, hk, 16, d // 2 + 4), 0xFF, np.uint8)
    return int4.kv_append_int4(empty, empty, bits(k), bits(v), slots, NAMES[k.dtype])


def check_weighted(q, k, v, scale, what=""):
    """One sequence: q [H][D], k / v [n][Hkv][D] (16-bit tensors)."""
    n, hk, d = k.shape
    nb = -(-n // 16)
    table = np.random.default_rng(n).permutation(nb).astype(np.int32)
    kp, vp = pools_of(k, v, table, nb)
    out = pkv.paged_decode_attention_int4(q[None].to(DEV), torch.from_numpy(kp).to(DEV), torch.from_numpy(vp).to(DEV),
                                          torch.from_numpy(table[None].copy()).to(DEV),
                                          torch.tensor([n], dtype=torch.int32, device=DEV), scale)
    pkv.paged_kv_check_status()
    got = widen_out(out.cpu(), NAMES[q.dtype])[0]
    q64 = widen_out(q, NAMES[q.dtype])
    K, V = (int4.values(p[table], f).transpose(0, 2, 1, 3).reshape(-1, hk, d)[:n] for p, f in ((kp, False), (vp, True)))
    pairs = np.ascontiguousarray(int4.tiles(vp[table])[:, :, 8 * d:]).view(np.float16).reshape(nb, hk, 16, 2)
    s = pairs[..., 0].astype(np.float64).transpose(0, 2, 1).reshape(-1, hk)[:n]
    g = q.shape[0] // hk
    u = torch.finfo(q.dtype).eps / 2
    w = torch.finfo(q.dtype).smallest_normal * u
    assert np.isfinite(got).all(), what
    for h in range(q.shape[0]):
        j = h // g
        x = K[:, j] @ q64[h] * scale
        p = np.exp(x - x.max())
        p /= p.sum()
        ref = p @ V[:, j]
        H = 7.5 * (p @ s[:, j])
        A = p @ np.abs(V[:, j]).max(-1)
        tol = (2.0 ** -11 + n * 2.0 ** -25) * H + 2.0 ** -13 * A + n * 2.0 ** -46 + u * np.abs(ref) + w
        err = np.abs(got[h] - ref)
        assert (err <= tol).all(), (what, h, float((err / tol).max()))


def context(n, d, dtype, seed, g=4, hk=2, spread=1.0):
    """Queries of a KV head that share a direction, keys and values N(0, 1)."""
    gen = torch.Generator().manual_seed(seed)
    base = torch.randn(hk, 1, d, generator=gen)
    q = (base + 0.5 * torch.randn(hk, g, d, generator=gen)).reshape(hk * g, d).to(dtype)
    k = (spread * torch.randn(n, hk, d, generator=gen)).to(dtype)
    v = torch.randn(n, hk, d, generator=gen)
    return gen, base[:, 0], q, k, v


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mag", [1e-3, 0.1, 1.0])
@pytest.mark.parametrize("n,at", [(600, [0]), (600, [333]), (600, [599]), (2048, list(range(5, 2048, 64))), (40, [3]),
                                  (2048, list(range(0, 2048, 2)))])
def test_rows_of_the_largest_range_without_weight(n, at, mag, d, dtype):
    """Rows of +-65504 whose keys point away from every query (weight below e^-35), beside rows of +-mag."""
    _, base, q, k, v = context(n, d, dtype, n + len(at))
    v = (mag * v).clamp(-3 * mag, 3 * mag)
    k[at] = (-8.0 * base).to(dtype)
    v[at] = 65504.0 * torch.where(torch.arange(d) % 2 == 0, 1.0, -1.0)
    x = torch.einsum("hgd,hd->hg", q.view(2, 4, d).float(), -8.0 * base) * d ** -0.5
    assert (x < -35).all()          # and the others' scores reach at least 0, their sum more
    check_weighted(q, k, v.to(dtype), d ** -0.5, f"{n} {len(at)} {mag}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [17, 300, 5000])
def test_scales_spread_over_the_whole_float16_range(n, d, dtype):
    """Rows of e^-14 .. e^9 in random order, ascending and descending, under sharp weights."""
    gen, _, q, k, v = context(n, d, dtype, n, spread=2.0)
    f = torch.empty(n, 2, 1).uniform_(-14, 9, generator=gen)
    for order in ("random", "up", "down"):
        e = f if order == "random" else f.sort(0, descending=order == "down").values
        check_weighted(q, k, (v * e.exp()).to(dtype), d ** -0.5, order)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("level", [0.0, 1e-4, 2.0])
def test_the_heaviest_rows_are_constant(level, d):
    """Rows of scale 0 carry nearly all of the weight (their products with the scale are 0)."""
    n, dtype = 500, torch.float16
    _, base, q, k, v = context(n, d, dtype, 3)
    k[::7] = (3.0 * base).to(dtype)
    v[::7] = level
    check_weighted(q, k, v.to(dtype), d ** -0.5)
    check_weighted(q, k, torch.full_like(v, level).to(dtype), d ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_with_a_nan_are_nan_and_alone(d, dtype):
    """Both appends store the same bytes for a row with a NaN; it reads and attends as NaN, its neighbours as ever."""
    hk, g, n, nb = 2, 3, 40, 6
    gen = torch.Generator().manual_seed(d)
    k, v = (torch.randn(n, hk, d, generator=gen).to(dtype) for _ in range(2))
    nan = float("nan")
    v[5, 1, 7], v[6, 0], k[21, 0, d - 1] = nan, nan, nan
    v[8, 1, :4] = torch.tensor([nan, float("inf"), -float("inf"), 1.0])
    v[9, 0, 3], v[10, 0, 5] = float("inf"), -float("inf")           # no NaN: limited, as ever
    k[22, 1].view(torch.int16)[9] = -1                              # a negative NaN
    table = np.array([3, 0, 5], np.int32)
    rk, rv = pools_of(k, v, table, nb)
    slots = (table[np.arange(n) // 16] * 16 + np.arange(n) % 16).astype(np.int32)
    kp, vp = (torch.full((nb, hk, 16, d // 2 + 4), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2))
    pkv.paged_kv_append_int4(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), kp, vp)
    assert np.array_equal(kp.cpu().numpy(), rk) and np.array_equal(vp.cpu().numpy(), rv)
    # the same rows one by one through the fused step
    k2, v2 = (torch.full_like(kp, 0xFF) for _ in range(2))
    bt = torch.from_numpy(table[None].copy()).to(DEV)
    q = torch.randn(1, hk * g, d, generator=gen).to(dtype).to(DEV)
    for i in range(n):
        cl = torch.tensor([i + 1], dtype=torch.int32, device=DEV)
        out = pkv.paged_decode_step_int4(q, k[i:i + 1].to(DEV), v[i:i + 1].to(DEV), k2, v2, bt, cl, 0.1)[0].float().cpu()
        ref = int4.decode_attention(widen_out(q.cpu(), NAMES[dtype]), rk, rv, table[None], [i + 1], 0.1)[0]
        assert np.array_equal(np.isnan(out.numpy()), np.isnan(ref)), i
        assert np.isnan(ref[:g]).all() == (i >= 6) and np.isnan(ref[g:]).all() == (i >= 5)
    assert torch.equal(k2, kp) and torch.equal(v2, vp)
    ko, vo = pkv.paged_kv_read_int4(torch.from_numpy(slots).to(DEV), kp, vp, dtype)
    pkv.paged_kv_check_status()
    assert torch.equal(ko.cpu().isnan().all(-1), k.isnan().any(-1)) and torch.equal(vo.cpu().isnan().any(-1), v.isnan().any(-1))
    assert torch.equal(ko.cpu().isnan().any(-1), k.isnan().any(-1)) and torch.equal(vo.cpu().isnan().all(-1), v.isnan().any(-1))


@pytest.mark.parametrize("at", [0, 9, 70, 299])
def test_a_nan_key_gives_nan_for_its_kv_head_alone(at):
    """Anywhere in a context, in the first step or a later one."""
    n, d, dtype = 300, 128, torch.bfloat16
    _, _, q, k, v = context(n, d, dtype, 5)
    k[at, 1, 3] = float("nan")
    nb = -(-n // 16)
    table = np.arange(nb, dtype=np.int32)
    kp, vp = pools_of(k, v.to(dtype), table, nb)
    out = pkv.paged_decode_attention_int4(q[None].to(DEV), torch.from_numpy(kp).to(DEV), torch.from_numpy(vp).to(DEV),
                                          torch.from_numpy(table[None].copy()).to(DEV),
                                          torch.tensor([n], dtype=torch.int32, device=DEV), 0.1)[0]
    pkv.paged_kv_check_status()
    assert out[4:].isnan().all() and torch.isfinite(out[:4]).all()
