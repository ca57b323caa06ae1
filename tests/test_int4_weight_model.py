"""CPU model of the 4-bit decode kernel's softmax reference (constants read from
the kernel source): products of weight and scale in float16 under a reference
that follows the largest product.  Rows that carry no weight must not cost the
others their low bits, whatever their scale."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_26_gb300", "csrc")
SRC = open(os.path.join(CSRC, "decode_int4.cuh")).read()


def const(name):
    return float(re.search(rf"constexpr \w+ {name} = (-?[\d.]+)f?;", SRC).group(1))


TOP, TARGET, SCALE_SLACK, STAGE = const("kTop"), const("kTarget"), const("kScaleSlack"), 16 * int(const("kBlocksPerStage"))
TINY = 2.0 ** -24


def attend(x, s, mid, dev, by_product=True):
    """Mean of mid + dev (dev = s (c - 7.5)) under weights 2^x; the largest float16
    product; how many steps looked at their products.  by_product False: the
    reference moves on the largest score and the largest scale apart."""
    M, cap, limit, l, b, acc, top, looked = 0.0, -1.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0
    for t in range(0, len(x), STAGE):
        xs, ss = x[t:t + STAGE] - M, s[t:t + STAGE]
        if xs.max() > limit or ss.max() > cap:
            looked += 1
            first, e = cap < 0, np.floor(np.log2(max(ss.max(), TINY)))
            if by_product or first or 2.0 ** e >= cap:
                cap, limit = 2.0 ** (e + SCALE_SLACK), TOP - (e + SCALE_SLACK)
            if by_product:
                d = (xs + np.floor(np.log2(np.maximum(ss, TINY)))).max() - TARGET
            else:
                d = xs.max() - (limit - (TOP - SCALE_SLACK))
            d = d if first else max(d, 0.0)
            M, xs = M + d, xs - d
            if not first:
                l, b, acc = l * 2.0 ** -d, b * 2.0 ** -d, acc * 2.0 ** -d
        p = 2.0 ** xs
        P = np.float16(p * ss).astype(np.float64)
        assert np.isfinite(P).all() and p.max() < 2.0 ** 60
        top = max(top, P.max())
        l += p.sum()
        b += (p * mid[t:t + STAGE]).sum()
        acc += (P / np.where(ss > 0, ss, 1.0) * dev[t:t + STAGE]).sum()
    return (acc + b) / l, top, looked


def draw(rng, n, s):
    dev = s * rng.choice(np.arange(16) - 7.5, n)
    return dev, 0.01 * s * rng.standard_normal(n)


def outlier(rng, n):
    """One row of +-65504 without weight beside rows of +-0.1."""
    x, s = 2 * rng.standard_normal(n), np.full(n, 0.0133)
    at = int(rng.integers(0, n))
    x[at], s[at] = -100.0, 8733.0
    return x, s


def spread(rng, n):
    return 4 * rng.standard_normal(n), np.float16(np.exp(rng.uniform(-14, 9, n))).astype(float)


def constants(rng, n):
    """Rows of scale 0 hold nearly all of the weight."""
    x, s = rng.standard_normal(n), np.full(n, 0.3)
    x[::7], s[::7] = 30.0, 0.0
    return x, s


def ordinary(rng, n):
    return 1.5 * rng.standard_normal(n), np.float16(0.33 * np.exp(0.15 * rng.standard_normal(n))).astype(float)


@pytest.mark.parametrize("kind", [outlier, spread, constants, ordinary], ids=lambda f: f.__name__)
@pytest.mark.parametrize("n", [1, 64, 65, 700, 4096])
def test_products_lose_half_a_step_of_their_own_weight(kind, n):
    rng = np.random.default_rng(n)
    for _ in range(20):
        x, s = kind(rng, n)
        dev, mid = draw(rng, n, s)
        got, top, looked = attend(x, s, mid, dev)
        p = 2.0 ** (x - x.max())
        p /= p.sum()
        want = (p * (mid + dev)).sum()
        H = 7.5 * (p * s).sum()
        # 2^-11 of each product, 2^-25 of those in float16's subnormal range (the largest is at least 1, or its row has
        # scale 0 and counts as 2^-24); sums here in 64 bits
        assert abs(got - want) <= (2.0 ** -11 + n * 2.0 ** -25) * H + n * 2.0 ** -46 + 1e-9 * abs(want)
        assert top < 2.0 ** TOP * 1.001
        if kind is ordinary:
            assert looked <= 2      # one vote a step, mostly


def test_the_largest_scale_alone_would_not_do():
    """The planted mistake: with the largest scale met, whatever its weight, the outlier breaks the bound."""
    rng = np.random.default_rng(0)
    worst = 0.0
    for _ in range(20):
        x, s = outlier(rng, 700)
        dev, mid = draw(rng, 700, s)
        got, _, _ = attend(x, s, mid, dev, by_product=False)
        p = 2.0 ** (x - x.max())
        p /= p.sum()
        worst = max(worst, abs(got - (p * (mid + dev)).sum()) / (2.0 ** -11 * 7.5 * (p * s).sum()))
    assert worst > 8


def test_the_oracle_keeps_a_nan_in_its_row():
    from oracle import int4
    x = np.linspace(-1, 1, 3 * 64, dtype=np.float32).reshape(3, 64)
    clean = int4.quantise_rows(x)
    x[1, 5] = np.nan
    codes, pairs = int4.quantise_rows(x)
    assert not codes[1].any() and list(pairs[1].view(np.uint16)) == [0, 0x7FFF]
    for i in (0, 2):
        assert np.array_equal(codes[i], clean[0][i]) and np.array_equal(pairs[i], clean[1][i])
