"""A 4-bit step of no sequences is nothing to do, as attention over none is
(no GPU needed)."""
import ctypes

import pytest

from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, lib


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def test_no_sequences():
    p, null = ctypes.c_void_p(4096), ctypes.c_void_p(0)
    d = PkvDims(0, 8, 2, 128, 16, 4, 2, 1)
    assert lib().paged_decode_attention_int4(null, p, p, null, null, 0.1, null, null, 0, ctypes.byref(d), null) == 0
    assert lib().paged_decode_step_int4(null, null, null, p, p, null, null, 0.1, null, null, 0, ctypes.byref(d), null) == 0
    d.num_seqs = 1
    assert lib().paged_decode_step_int4(p, null, null, p, p, p, p, 0.1, p, p, 0, ctypes.byref(d), null) == -1
    assert lib().paged_decode_step_int4(p, null, null, p, p, p, p, 0.1, p, p, 0, None, null) == -1
