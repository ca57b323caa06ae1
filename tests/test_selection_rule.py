"""CPU: the selection's oracle and the plain form of perf/more_operators.py follow one rule
where queries are not finite: the head's scale is not finite either, its codes are 0, and
0 times that, a NaN, counts as +infinity."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import long_context as lc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SPEC = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan, 3e38])
def test_one_head_beside_finite_ones(value):
    plain = importlib.util.module_from_spec(SPEC)
    SPEC.loader.exec_module(plain)
    rng = np.random.default_rng(0)
    bounds = np.sort(rng.integers(-127, 128, (20, 1, 2, 64)).astype(np.int8), axis=2)[:, :, ::-1].copy()
    scales = rng.random((20, 1)).astype(np.float32)
    q = torch.from_numpy(rng.normal(size=(1, 4, 64))).bfloat16()
    q[0, 2, 5] = float(value)
    tables, lens = np.arange(20, dtype=np.int32)[None], [320]
    got = lc.select_blocks(q.float().numpy(), bounds, scales, tables, lens, 6, 1, 1)
    want = plain._select(q, torch.from_numpy(bounds), torch.from_numpy(scales), torch.from_numpy(tables),
                         torch.tensor(lens), 6, 1, 1)
    assert np.array_equal(got, want.numpy())
    if not np.isfinite(value):
        assert got.tolist() == [[[0, 1, 2, 3, 4, 19]]]
