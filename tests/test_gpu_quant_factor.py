"""Factors that are not finite: reported, and their matrices are zero."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q
from quant_utils import DEV, random_weights, status, to64, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("kind,group", [("e2m1", 16), ("int4", 32)])
def test_a_factor_that_is_not_finite(kind, group, bad):
    rng = np.random.default_rng(3)
    codes, scales, factors = random_weights(rng, 3, 130, 264, kind, group)
    factors[1] = bad
    d = B.QuantDesc(3, 130, 264, kind, group)
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_pack(d, *(torch.from_numpy(v).to(DEV) for v in (codes, scales, factors)), packed, st))
    assert B.moe_get_device_status(st) == 6
    factors[1] = 0
    want = Q.weights(codes, scales, factors, kind, group)
    w = torch.full((3, 130, 264), float("nan"), dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_unpack(d, packed, w))
    assert (to64(w)[1] == 0).all()
    # the product with the factor rounded to fp32, then to bf16
    assert (np.abs(to64(w) - want) <= np.abs(want) * (2.0 ** -24 + Q.STEP)).all()


@pytest.mark.parametrize("T", [2, 8, 20, 80])
def test_products_with_such_a_matrix_are_zero(T):
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.normal(size=(T, 264))).to(DEV, torch.bfloat16)
    for swiglu in (False, True):
        w = random_weights(rng, 1 + swiglu, 96, 264, "e2m1", 16)
        w[2][-1] = float("inf")                  # the only matrix, or `up`
        q = B.QuantDesc(1 + swiglu, 96, 264, "e2m1", 16)
        packed, st = torch.empty(B.moe_quant_size(q), dtype=torch.uint8, device=DEV), status()
        B.check(B.moe_quant_pack(q, *(torch.from_numpy(v).to(DEV) for v in w), packed, st))
        assert B.moe_get_device_status(st) == 6
        d = B.QuantProject(T, 264, 96 * (1 + swiglu), "e2m1", 16, swiglu)
        y, ws = torch.full((T, 96), 7.0, dtype=torch.bfloat16, device=DEV), torch.empty(256, dtype=torch.uint8, device=DEV)
        B.check(B.moe_quant_project(d, x, packed, y, st, ws))
        torch.cuda.synchronize()
        assert (y == 0).all()


def test_the_rest_of_a_layer_with_such_an_expert():
    """One expert's down matrix has no factor: its share of the sum is zero, the others' stay."""
    T, H, E, I, k = 20, 192, 4, 64, 2  # noqa: E741
    rng = np.random.default_rng(9)
    raw = [random_weights(rng, n, r, c, "int4", 16) for n, r, c in ((2 * E, I, H), (E, H, I))]
    raw[1][2][3] = float("nan")
    packed = []
    st = status()
    for w in raw:
        q = B.QuantDesc(w[0].shape[0], w[0].shape[1], 2 * w[0].shape[2], "int4", 16)
        packed.append(torch.empty(B.moe_quant_size(q), dtype=torch.uint8, device=DEV))
        B.check(B.moe_quant_pack(q, *(torch.from_numpy(v).to(DEV) for v in w), packed[-1], st))
    assert B.moe_get_device_status(st) == 6
    st.zero_()
    token = np.arange(T * k, dtype=np.int32) % T
    offsets = np.array([0, 5, 11, 19, T * k], dtype=np.int32)
    x = torch.from_numpy(rng.normal(size=(T, H))).to(DEV, torch.bfloat16)
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=k)
    y = torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    B.check(B.moe_grouped_ffn_quant(d, B.QuantWeights("int4", 16, *packed), x, torch.from_numpy(token).to(DEV),
                                    torch.from_numpy(offsets).to(DEV), y, st, ws))
    assert B.moe_get_device_status(st) == 0
    raw[1][2][3] = 0
    gu, dn = (Q.weights(*w, "int4", 16) for w in raw)
    x64 = to64(x)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        within(y[a:b], *Q.ffn(x64[token[a:b]], gu[2 * e], gu[2 * e + 1], dn[e]), f"expert {e}")
    assert (y[offsets[3]:] == 0).all()
