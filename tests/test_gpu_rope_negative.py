"""GPU: negative frequencies turn the other way, tiny ones not at all (bound: test_gpu_rope.bound)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, i32, rand
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build
from test_gpu_rope import bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_frequencies(dtype, interleaved):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    inv = [-1.0, 0.5, -1e-20, -1e-6, 1e-3, -3.7, -5e-324, -2.0 ** -54]
    pos = np.array([0, 1, -1, 77, 1 << 20, -(1 << 20)])
    q, k = rand((6, 2, 64), dtype, 1), rand((6, 1, 64), dtype, 2)
    rope = pkv.make_rope(inv, 64, interleaved=interleaved)
    out = pkv.paged_kv_rope(q.to(DEV), k.to(DEV), i32(pos), rope)
    for x, got in zip((q, k), out):
        ref = lc.rope(f64(x), pos, inv, interleaved=interleaved)
        assert_within(f64(got), ref, bound(x, pos, inv, dtype, interleaved, 1.0, ref))
    # the mirrored frequencies at the mirrored positions: the same bits
    mirrored = pkv.paged_kv_rope(q.to(DEV), k.to(DEV), i32(-pos), pkv.make_rope([-f for f in inv], 64, interleaved=interleaved))
    assert torch.equal(out[0], mirrored[0]) and torch.equal(out[1], mirrored[1])
    pkv.paged_kv_check_status()
