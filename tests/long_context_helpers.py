"""Shared pieces of the GPU tests of rotary positions, chunk attention and block-sparse
decode: ragged paged inputs, and the bound that their outputs are held to."""
import numpy as np
import torch

DEV = "cuda"


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(dtype)


def paged(lens, seed=0, extra=3, width=None):
    """(tables numpy [B][W] with -1 behind the blocks, number of blocks): scattered."""
    nblk = [-(-int(n) // 16) for n in lens]
    nb = sum(nblk) + extra
    perm = np.random.default_rng(seed).permutation(nb)
    tables = np.full((len(lens), width or max([1, *nblk])), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
    return tables, nb


def hide_tails(pool, tables, lens, value=float("nan")):
    """Fills every slot that holds no token with `value`, unused blocks too."""
    used = np.zeros((pool.shape[0], 16), bool)
    for b, n in enumerate(lens):
        for j in range(-(-int(n) // 16)):
            used[tables[b, j], :min(16, int(n) - 16 * j)] = True
    pool.transpose(1, 2)[torch.from_numpy(~used)] = value
    return pool


def tolerance(ref, mag, dtype, q, k, v, scale, keys, weight_bits=None):
    """Elementwise bound of attention against 64 bits.

    u = eps/2 of the type (the output's one rounding; below the smallest normal value
    half a subnormal step, w).  A weight is rounded once to the type (relative u; with
    weight_bits given 2^-weight_bits), in fp16 by at most 2^-25 where it is subnormal
    beside a largest weight of 1 or more: the mean moves by u mean|v|, or keys 2^-25
    max|v|.  A logit is a float32 sum of D products: each of the D additions rounds, by
    2^-23 of the sum of magnitudes S at most (a tensor core may cut instead of
    rounding); its scaling and the reference add two roundings of a number below 1.5 S;
    exp2 is good to 2^-22.  A weight's relative error counts in the mean and in its
    normaliser.  Sums of `keys` weights in float32: 2^-24 keys, counted likewise
    (products with V accumulate so too)."""
    u = torch.finfo(dtype).eps / 2
    w = torch.finfo(dtype).smallest_normal * u
    S = abs(scale) * float(np.abs(q).max()) * float(np.abs(k[np.isfinite(k)]).max(initial=0)) * q.shape[-1]
    # the largest sum of magnitudes is far below the product of maxima: take Cauchy-Schwarz of the largest rows
    kn = np.sqrt((np.where(np.isfinite(k), k, 0) ** 2).sum(-1)).max(initial=0)
    S = min(S, abs(scale) * float(np.sqrt((q ** 2).sum(-1)).max()) * float(kn))
    e = 2.0 ** -23 * (q.shape[-1] + 3) * S + 2.0 ** -22 + 2.0 ** -24 * keys
    wu = u if weight_bits is None else 2.0 ** -weight_bits
    sub = keys * 2.0 ** -25 * float(np.abs(v[np.isfinite(v)]).max(initial=0)) if dtype == torch.float16 else 0.0
    return u * np.abs(ref) + w + (wu + 2 * e) * mag + sub


def assert_within(got, ref, tol, what=""):
    assert got.shape == ref.shape
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))           # infinities and NaN where they belong
    with np.errstate(invalid="ignore"):                                # (infinity less infinity)
        bad = ~same & ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], float(np.nanmax((np.abs(got - ref) / tol)[~same])))
