"""The float64 form of 4-bit weights against hand-computed values, and the words
that the library packs them into (layout only: no GPU)."""
import numpy as np
import pytest
import torch

from oracle import quant as Q


def test_values_by_hand():
    codes = np.array([[[0x71, 0xF8, 0x2A, 0x03]]], dtype=np.uint8)   # K 8: 1 7 8 f a 2 3 0
    scales = np.array([[[0x38]]], dtype=np.uint8)                    # 1.0
    w = Q.weights(codes, scales, [2.0], "e2m1", 16)
    assert w.tolist() == [[[1.0, 12.0, -0.0, -12.0, -2.0, 2.0, 3.0, 0.0]]]
    w = Q.weights(codes, scales, [0.5], "int4", 16)
    assert w.tolist() == [[[-3.5, -0.5, 0.0, 3.5, 1.0, -3.0, -2.5, -4.0]]]


def test_scales_are_e4m3():
    bits = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    got = Q.e4m3(bits)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


@pytest.mark.parametrize("group", [16, 32])
def test_groups_follow_the_inputs(group):
    K = 72                                             # the last group is cut
    n = -(-K // group)
    codes = np.full((1, 1, K // 2), 0x99, dtype=np.uint8)            # int 1
    scales = (0x38 + 8 * np.arange(n, dtype=np.uint8)).reshape(1, 1, n)
    w = Q.weights(codes, scales, [1.0], "int4", group)[0, 0]
    assert w.tolist() == [2.0 ** (k // group) for k in range(K)]


def test_products_by_hand_and_bounds():
    x, w = np.array([[1.0, 2.0]]), np.array([[3.0, -4.0]])
    y, d = Q.product(x, w)
    assert y.tolist() == [[-5.0]] and d[0, 0] == 6 * 2.0 ** -23 * 11
    y, d = Q.product(x, w, np.array([[0.5, 0.0]]))
    assert d[0, 0] == 6 * 2.0 ** -23 * 11 + 1.5
    y, _ = Q.ffn(np.array([[2.0]]), np.array([[1.0]]), np.array([[3.0]]), np.array([[0.5]]))
    assert abs(y[0, 0] - 0.5 * 6.0 * 2.0 / (1 + np.exp(-2.0))) < 1e-15
