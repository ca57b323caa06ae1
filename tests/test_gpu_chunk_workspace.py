"""GPU: one workspace of chunk attention for other batches and other layouts of heads of the
same head_dim, with units that are cut."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, hide_tails, i32, paged, rand, tolerance
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_shared_by_batches_and_heads(d):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    calls = [([40], [3000], 8, 2, torch.bfloat16), ([3, 300, 1], [2000, 700, 4097], 6, 6, torch.bfloat16),
             ([7, 9], [12, 9], 4, 1, torch.float16), ([600], [1300], 8, 1, torch.float16), ([40], [3000], 8, 2, torch.bfloat16)]
    ws, outs, checks = None, [], []
    for i, (new, lens, hq, hk, dtype) in enumerate(calls):
        tables, nb = paged(lens, i)
        kp, vp = (hide_tails(rand((nb, hk, 16, d), dtype, x + hk), tables, lens) for x in (1, 2))
        q, off = rand((sum(new), hq, d), dtype, 3), np.concatenate([[0], np.cumsum(new)])
        args = [x.to(DEV) for x in (q, kp, vp)] + [i32(tables), i32(lens), i32(off)]
        if ws is None:
            ws = pkv.make_workspace_chunk(args[0], args[1], args[3])
        checks.append((q, kp, vp, tables, lens, off))
        outs.append((args, torch.empty_like(args[0])))
    for args, out in outs:                                     # without a wait between them
        pkv.paged_chunk_attention(*args, 0.1, out=out, workspace=ws)
    pkv.paged_kv_check_status()
    for (q, kp, vp, tables, lens, off), (_, out) in zip(checks, outs):
        ref, mag = lc.chunk_attention(f64(q), f64(kp), f64(vp), tables, lens, off, 0.1)
        assert_within(f64(out), ref, tolerance(ref, mag, q.dtype, f64(q), f64(kp), f64(vp), 0.1, max(lens)))
