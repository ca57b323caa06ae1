"""Block copies: element sizes that are not one of the pools' are refused before
anything is launched (no GPU needed)."""
import ctypes
import os
import re

import pytest

from paged_kv_cache_26_gb300 import api
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, lib


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def copy(elem, pairs=1):
    p = ctypes.c_void_p(1 << 20)
    d = PkvDims(0, 8, 8, 128, 16, 10, 0, 1)
    return lib().paged_kv_copy_blocks(p, p, p, pairs, ctypes.byref(d), elem, ctypes.c_void_p(0))


def test_element_sizes():
    header = open(os.path.join(pkv_build.INCLUDE, "paged_kv.h")).read()
    assert int(re.search(r"PKV_ELEM_INT4 = (-?\d+)", header).group(1)) == api.PKV_ELEM_INT4
    for elem in (0, 3, 4, 8, -1, -2):          # 0: a size that was never set
        assert copy(elem) == -1, elem
    for elem in (1, 2, api.PKV_ELEM_INT4):
        assert copy(elem, pairs=0) == 0
