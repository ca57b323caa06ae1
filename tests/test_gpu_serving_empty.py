"""Resize and verification with empty arguments."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


@pytest.mark.parametrize("width", [4, 4000])       # one CTA, and a cluster
def test_a_slot_map_without_room_takes_no_tokens(width):
    tables = np.full((3, width), -1)
    tables[0, 0], tables[1, :2] = 5, (7, 3)
    before = [i32([16, 20, 0]), i32(tables), i32([9, 8, 6, -1, -1, -1, -1, -1, -1, -1]), i32([3])]
    room = i32(np.zeros(4))
    for new, ok in (([18, 20, 0], False), ([16, 20, 1], False), ([0, 21, 0], False), ([16, 17, 0], True), ([3, 1, 0], True),
                    ([16, 20, 0], True)):
        d = [t.clone() for t in before]
        slots, offs = room[:0], i32([7, 7, 7, 7])
        pkv.paged_kv_resize_tables(d[0], i32(new), d[1], d[2], d[3], slots, offs)
        assert offs.tolist() == [0, 0, 0, 0]
        if ok:
            pkv.paged_kv_check_status()
            assert d[0].tolist() == new
        else:
            with pytest.raises(pkv.PagedKVError) as e:
                pkv.paged_kv_check_status()
            assert e.value.code == -6
            assert all(torch.equal(a, b) for a, b in zip(d, before))
    # without a map any growth is taken
    d = [t.clone() for t in before]
    pkv.paged_kv_resize_tables(d[0], i32([18, 20, 0]), d[1], d[2], d[3])
    pkv.paged_kv_check_status()
    assert d[0].tolist() == [18, 20, 0] and d[1][0, 1] == 6


@pytest.mark.parametrize("by_stream", [False, True])
def test_an_empty_batch_has_lengths_when_it_gave_some(by_stream):
    t, d = torch.zeros(0, 3, 8, device=DEV), torch.zeros(0, 2, 8, device=DEV)
    x, au, su = torch.zeros(0, 2, dtype=torch.int32, device=DEV), torch.zeros(0, 2, device=DEV), torch.zeros(0, device=DEV)
    stream = torch.cuda.Stream() if by_stream else None
    a, out, lens = pkv.paged_verify_draft(t, d, x, au, su, context_lens=i32([]), stream=stream)
    assert a.shape == (0,) and out.shape == (0, 3) and lens.shape == (0,) and lens.dtype == torch.int32
    assert pkv.paged_verify_draft(t, d, x, au, su, stream=stream)[2] is None
    free, num = i32([0, 1]), i32([2])
    pkv.paged_kv_resize_tables(i32([]), lens, i32(np.zeros((0, 4))), free, num)   # and on to giving back
    pkv.paged_kv_check_status()
