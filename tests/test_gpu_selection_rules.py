"""GPU: queries that are not finite in the selection of blocks, and lists of empty sequences
in the attention over them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, i32, paged, rand
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 2), (3, 1), (10, 2), (16, 2)])
@pytest.mark.parametrize("width", [64, 300, 2500])  # scores and choice in one launch, and in two of either kind
def test_queries_that_are_not_finite(dtype, d, hq, hk, width):
    """One head with an infinity or NaN beside finite ones: every block's score is +infinity, the lowest are chosen."""
    lens = [width * 16, 1000, 970, 1024]
    tables, nb = paged(lens, 5)
    rng = np.random.default_rng(width)
    bounds = np.sort(rng.integers(-127, 128, (nb, hk, 2, d)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.choice(np.float32([0.25, 0.5, 1e-3, 0.0, np.inf]), (nb, hk))
    q = rand((4, hq, d), DT[dtype], 6, 3.0)
    for b, value in ((0, np.inf), (1, -np.inf), (2, np.nan)):
        q[b, hq - 1, 7 * b] = float(value)
    for num, sink, recent in ((6, 1, 1), (20, 0, 3)):
        got = pkv.paged_select_blocks(q.to(DEV), torch.from_numpy(bounds).to(DEV), torch.from_numpy(scales).to(DEV),
                                      i32(tables), i32(lens), num, sink, recent).cpu().numpy()
        pkv.paged_kv_check_status()
        assert np.array_equal(got, lc.select_blocks(q.float().numpy(), bounds, scales, tables, lens, num, sink, recent))
        for b in range(3):
            n = -(-lens[b] // 16)
            assert got[b, hk - 1].tolist() == [*range(num - recent), *range(n - recent, n)]


def test_lists_of_empty_sequences_are_flagged():
    """A listed block at or behind the context, of a sequence without tokens too."""
    lens = [0, 40]
    tables, nb = paged(lens, 1)
    kp, vp, q = rand((nb, 2, 16, 64), torch.bfloat16, 1), rand((nb, 2, 16, 64), torch.bfloat16, 2), rand((2, 4, 64), torch.bfloat16, 3)

    def attend(sel, tab=tables):
        return pkv.paged_decode_attention_sparse(q.to(DEV), kp.to(DEV), vp.to(DEV), i32(tab), i32(lens), i32(sel), 0.125)

    quiet = np.array([[[-1, -1]] * 2, [[0, 2]] * 2])
    want = attend(quiet)
    pkv.paged_kv_check_status()
    assert not want[0].any()
    for entry in (0, 1, 7, 2 ** 31 - 1):
        sel = quiet.copy()
        sel[0, 1, 1] = entry
        got = attend(sel)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == -6 and torch.equal(got, want)
        pkv.paged_kv_check_status()
