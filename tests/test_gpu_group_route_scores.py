"""Scores that the selection compares: a sigmoid is within 1e-6 of its own value, so
units whose scores differ by 2e-6 of them and more come out in order, however small
the scores are."""
import numpy as np
import pytest
import torch
from test_gpu_group_route import _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ulps,low,high", [(4, 8, 15), (2, 16, 31), (1, 33, 63), (1, 65, 85)])
@pytest.mark.parametrize("groups", [1, 4, 64])
def test_neighbouring_logits_far_below_zero_come_out_in_order(ulps, low, high, groups):
    """Of each token one pair of units, `ulps` steps of fp32 apart, is far above the
    rest; equal scores would go to the lower unit, so the higher one has the larger."""
    T, E = 2000, 128
    rng = np.random.default_rng(low + groups)
    l = np.full((T, E), -100.0, dtype=np.float32)
    a = -rng.uniform(low, high, T).astype(np.float32)
    b = a.copy()
    for _ in range(ulps):
        b = np.nextafter(b, np.float32(0))
    u = np.sort(np.argsort(rng.random((T, E)), axis=1)[:, :2], axis=1)
    l[np.arange(T), u[:, 0]], l[np.arange(T), u[:, 1]] = a, b
    gap = 1 - np.exp(a.astype(np.float64) - b)
    assert (gap >= 2e-6).all()
    kt = np.full(T, 2, dtype=np.int32)
    out = _run(l, None, kt, 2, groups, groups, 1, "sigmoid", True)
    got = out[0] if isinstance(out[0], np.ndarray) else out[0].cpu().numpy()
    assert (got == u[:, ::-1]).all()


@pytest.mark.parametrize("groups", [1, 64])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_at_the_ends_of_fp32(groups, score):
    """Of a lowest value that masks, not -inf, and of logits whose products overflow:
    in order, equal scores to the lower unit."""
    l = np.full((3, 128), np.finfo(np.float32).min, dtype=np.float32)
    l[0, [9, 20, 33]] = [2e38, 3e38, 5.0]
    l[1, [7, 8]] = [-1e38, -3e38]
    out = _run(l, None, np.full(3, 4, np.int32), 4, groups, groups, 1, score, True)
    if score == "sigmoid":      # 1, 1, 0.993, 0; the others are all 0
        assert list(out[0][0]) == [9, 20, 33, 0] and list(out[0][1]) == [0, 1, 2, 3]
    else:                       # one unit has it all
        assert out[0][0][0] == 20 and out[0][1][0] == 7
    assert list(out[0][2]) == [0, 1, 2, 3]
    w = out[1]
    assert np.isfinite(w).all() and np.allclose(w.sum(1), 2.5, rtol=1e-5)
