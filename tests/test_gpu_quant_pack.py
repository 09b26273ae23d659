"""Packing 4-bit weights: what is unpacked is the weights, to one rounding."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q
from quant_utils import DEV, pack, random_weights, status, to64

pytestmark = pytest.mark.gpu
KINDS = [("e2m1", 16), ("e2m1", 32), ("int4", 16), ("int4", 32)]


def _unpack(desc, packed):
    w = torch.full((desc.count, desc.rows, desc.K), float("nan"), dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_unpack(desc, packed, w))
    return w


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("count,rows,K", [(1, 1, 8), (3, 130, 264), (2, 128, 128), (5, 64, 40), (1, 257, 1000)])
def test_round_trip(kind, group, count, rows, K):
    rng = np.random.default_rng(rows + K)
    w = random_weights(rng, count, rows, K, kind, group)
    got = to64(_unpack(B.QuantDesc(count, rows, K, kind, group), pack(w, kind, group)))
    want = Q.weights(*w, kind, group)
    # fp32 code times scale is exact, its product with the factor rounded to fp32, then to bf16
    assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -24 + Q.STEP)).all()


@pytest.mark.parametrize("kind,group", KINDS)
def test_every_code_and_scale_is_exact(kind, group):
    """All 16 codes under all 127 scales, factor 1: code * scale has seven bits at most."""
    codes = np.zeros((1, 127, 64), dtype=np.uint8)
    codes[...] = np.tile(np.arange(0, 256, 17, dtype=np.uint8), 4)[None, None, :] & 0x0F
    codes |= (np.tile(np.roll(np.arange(16), 5), 4).astype(np.uint8) << 4)[None, None, :]
    n = -(-128 // group)
    scales = np.repeat(np.arange(127, dtype=np.uint8)[None, :, None], n, axis=2)
    w = (codes, scales, np.ones(1, dtype=np.float32))
    got = to64(_unpack(B.QuantDesc(1, 127, 128, kind, group), pack(w, kind, group)))
    assert np.array_equal(got, Q.weights(*w, kind, group))


@pytest.mark.parametrize("kind,group", KINDS)
def test_bad_scales_are_reported(kind, group):
    rng = np.random.default_rng(0)
    for byte, bad in ((0x7F, True), (0xFF, True), (0xB8, True), (0x80, False)):
        codes, scales, factors = random_weights(rng, 1, 4, 64, kind, group)
        scales[0, 2, 0] = byte
        d = B.QuantDesc(1, 4, 64, kind, group)
        t = [torch.from_numpy(v).to(DEV) for v in (codes, scales, factors)]
        packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
        B.check(B.moe_quant_pack(d, *t, packed, st))
        assert B.moe_get_device_status(st) == (6 if bad else 0)
        scales[0, 2, 0] = 0
        want = Q.weights(codes, scales, factors, kind, group)
        assert (np.abs(to64(_unpack(d, packed)) - want) <= np.abs(want) * (2.0 ** -24 + Q.STEP)).all()
    st = status()
    t[2][0] = float("inf")
    B.check(B.moe_quant_pack(d, *t, packed, st))
    assert B.moe_get_device_status(st) == 6


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("count,rows,K", [(2, 130, 264), (1, 3, 8), (4, 64, 512)])
def test_quantize(kind, group, count, rows, K):
    rng = np.random.default_rng(K)
    w = torch.from_numpy(rng.normal(size=(count, rows, K)) * K ** -0.5).to(DEV, torch.bfloat16)
    w[0, 0] = 0
    d = B.QuantDesc(count, rows, K, kind, group)
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_quantize(d, w, packed, st))
    assert B.moe_get_device_status(st) == 0
    w64, got = to64(w), to64(_unpack(d, packed))
    assert (got[0, 0] == 0).all()
    n = -(-K // group)
    pad = np.zeros((count, rows, n * group))
    pad[..., :K] = np.abs(w64)
    amax = np.repeat(pad.reshape(count, rows, n, group).max(3), group, axis=2)[..., :K]
    vmax = 7.0 if kind == "int4" else 6.0
    # The scale is within 2^-4 of amax / vmax (half an e4m3 step, or of the smallest one,
    # 2^-10 / 448 of the matrix's largest), a code within half its widest gap (int 1/2; e2m1 1)
    # or, where the scale fell short, the largest code off by what is missing.
    tiny = np.abs(w64).max((1, 2), keepdims=True) * 2.0 ** -10 / 448 / vmax
    scale = amax / vmax * (1 + 2.0 ** -4) + tiny
    gap = 0.5 if kind == "int4" else 1.0
    lim = gap * scale + amax * 2.0 ** -4 + vmax * tiny + np.abs(w64) * 2 * Q.STEP
    assert (np.abs(got - w64) <= lim).all()
    # bell-shaped weights lose about a tenth of their norm in 4 bits
    assert np.linalg.norm(got - w64) < 0.13 * np.linalg.norm(w64)


def test_quantize_reports_what_is_not_finite():
    d = B.QuantDesc(1, 4, 64, "e2m1", 16)
    w = torch.ones(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    w[0, 1, 3], w[0, 2, 5] = float("inf"), float("nan")
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_quantize(d, w, packed, st))
    assert B.moe_get_device_status(st) == 6
    got = _unpack(d, packed)
    assert got[0, 1, 3] == 0 and got[0, 2, 5] == 0 and (got == 1).sum() == 4 * 64 - 2


@pytest.mark.parametrize("kind,group", KINDS)
def test_quantize_weights_near_the_smallest(kind, group):
    """Largest weight 2^-120: the groups' steps are subnormal, their reciprocals infinite."""
    w = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device=DEV)
    w[0, 0, 0] = 2.0 ** -120
    w[0, 1, ::2] = 2.0 ** -127
    d = B.QuantDesc(1, 3, 64, kind, group)
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_quantize(d, w, packed, st))
    assert B.moe_get_device_status(st) == 0
    got = _unpack(d, packed)
    assert ((got == 0) == (w == 0)).all()
    # the factor (2^-131) has 18 bits, a scale off by up to 2^-4, a product rounded to a bf16
    # subnormal (2^-134, 2^-7 of 2^-127)
    assert (np.abs(to64(got) - to64(w)) <= (2.0 ** -4 + 2.0 ** -7 + 2.0 ** -17) * np.abs(to64(w))).all()
