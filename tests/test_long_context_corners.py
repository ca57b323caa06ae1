"""CPU pins of oracle/long_context.py where logits are -infinity."""
import numpy as np

from oracle import long_context as lc


def test_rows_of_minus_infinity_are_nan_and_rows_without_keys_zero():
    rng = np.random.default_rng(0)
    k, v, q = (rng.normal(size=(n, 8)) for n in (6, 6, 4))
    q[:, 0] = 1.0
    k[:3, 0] = -np.inf
    seen = np.array([[0] * 6, [1, 1, 0, 0, 0, 0], [1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 1]], bool)
    out, mag = lc.attend(q, k, v, seen, 0.5)
    assert not out[0].any() and np.isnan(out[1:3]).all() and np.isnan(mag[1:3]).all()
    alone, _ = lc.attend(q[3:], k[[3, 5]], v[[3, 5]], np.ones((1, 2), bool), 0.5)
    assert np.allclose(out[3], alone[0])
    # softmax by its definition
    with np.errstate(invalid="ignore"):
        s = (q[2] @ k[:3].T) * 0.5
        e = np.exp(s - s.max())
        assert np.isnan(e / e.sum()).all()
