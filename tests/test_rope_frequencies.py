"""CPU: the frequencies of rotary positions as turns in units of 2^-64: negative ones are the
negatives, whatever their size, and factors that no float32 holds are refused."""
import ctypes

import pytest

from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvRope, lib

INVALID = -1


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def init(freqs, factor=1.0):
    r, n = PkvRope(), len(freqs)
    rc = lib().paged_kv_rope_init(ctypes.byref(r), (ctypes.c_double * n)(*freqs), n, None, 1, 0, factor)
    return rc, r


def test_negative_frequencies():
    freqs = [1.0, 0.75, 1e-3, 1e-9, 1e-20, 5e-324, 6.5, 1e6, 1e-6, 2.0 ** -54, 3.14159265358979, 1e12, 0.0, 100.25, 1e-17, 7e15]
    rc, up = init(freqs)
    assert rc == 0
    rc, down = init([-f for f in freqs])
    assert rc == 0
    for f in range(len(freqs)):
        assert down.turns[f] == -up.turns[f] % 2 ** 64, freqs[f]
    # the smallest ones are nothing at all, not half a turn or nearly a whole one beside nothing
    assert up.turns[5] == 0 and up.turns[4] == down.turns[4] == 0 and up.turns[12] == 0


@pytest.mark.parametrize("factor,ok", [(1e39, False), (-1e300, False), (3.4e38, True), (-2.0, True), (0.0, True), (1e-50, True),
                                       (float("inf"), False), (float("nan"), False)])
def test_factors(factor, ok):
    assert init([1.0] * 8, factor)[0] == (0 if ok else INVALID)
