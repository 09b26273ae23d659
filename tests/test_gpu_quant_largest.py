"""4-bit calls at the ends of what they accept: 2^23 tokens, more matrices than a grid has rows,
2^20 outputs and inputs, experts split into units."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q
from quant_utils import DEV, Layer, pack, random_weights, status, to64, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("swiglu", [False, True])
def test_the_most_tokens(swiglu):
    T, K, N, halves = 1 << 23, 72, 258, 1 + swiglu
    w = random_weights(np.random.default_rng(1), halves, N // halves, K, "e2m1", 16)
    x = torch.randn(T, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).bfloat16()
    y, st = torch.full((T + 1, N // halves), 7.0, dtype=torch.bfloat16, device=DEV), status()
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    B.check(B.moe_quant_project(B.QuantProject(T, K, N, "e2m1", 16, swiglu), x, pack(w, "e2m1", 16), y, st, ws))
    assert B.moe_get_device_status(st) == 0 and (y[T:] == 7.0).all()
    w64 = Q.weights(*w, "e2m1", 16)
    for rows in (slice(0, 200), slice(T // 2 - 100, T // 2 + 100), slice(T - 300, T)):
        x64 = to64(x[rows])
        within(y[rows], *(Q.swiglu(*Q.product(x64, w64[0]), *Q.product(x64, w64[1])) if swiglu
                          else Q.product(x64, w64[0])))


@pytest.mark.parametrize("kind,group", [("e2m1", 16), ("int4", 32)])
def test_more_matrices_than_a_grid_has_rows(kind, group):
    count, rows, K = 70000, 3, 24
    rng = np.random.default_rng(2)
    codes = torch.from_numpy(rng.integers(0, 256, (count, rows, K // 2), dtype=np.uint8)).to(DEV)
    scales = torch.from_numpy(rng.integers(0x30, 0x44, (count, rows, -(-K // group)), dtype=np.uint8)).to(DEV)
    factors = torch.rand(count, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)) + 0.5
    d = B.QuantDesc(count, rows, K, kind, group)
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_pack(d, codes, scales, factors, packed, st))
    w = torch.full((count, rows, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_unpack(d, packed, w))
    assert B.moe_get_device_status(st) == 0
    want = Q.weights(codes.cpu().numpy(), scales.cpu().numpy(), factors.cpu().numpy(), kind, group)
    # the product with the factor rounded to fp32, then to bf16
    assert (np.abs(to64(w) - want) <= np.abs(want) * (2.0 ** -24 + Q.STEP)).all()
    # Quantised, each matrix has its own factor, top / (448 v_max) rounded: its largest weight gets
    # the scale 448 and the largest code, so it comes back to the factor's rounding and bf16's.
    top = w.abs().flatten(1).max(1)[0].double()
    B.check(B.moe_quant_quantize(d, w, packed, st))
    back = torch.full_like(w, float("nan"))
    B.check(B.moe_quant_unpack(d, packed, back))
    assert B.moe_get_device_status(st) == 0
    off = (back.abs().flatten(1).max(1)[0].double() - top).abs()
    assert (off <= top * (2.0 ** -8 + 2.0 ** -22)).all()


@pytest.mark.parametrize("T", [2, 8, 40])
def test_the_longest_sums_and_the_widest_outputs(T):
    """K 2^20 with N 40, then N 2^20 with K 40."""
    for K, N in ((1 << 20, 40), (40, 1 << 20)):
        w = random_weights(np.random.default_rng(T), 1, N, K, "int4", 32)
        x = torch.randn(T, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).bfloat16()
        y, st = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV), status()
        ws = torch.empty(256, dtype=torch.uint8, device=DEV)
        B.check(B.moe_quant_project(B.QuantProject(T, K, N, "int4", 32), x, pack(w, "int4", 32), y, st, ws))
        assert B.moe_get_device_status(st) == 0
        within(y, *Q.product(to64(x), Q.weights(*w, "int4", 32)[0]))


@pytest.mark.parametrize("T", [1, 8, 30])
def test_experts_split_into_units(T):
    """8 experts of 4 units each, a bias an expert: the layer against its own routing."""
    layer = Layer(T, 256, 32, 64, "e2m1", 16)
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.normal(size=(T, 256))).to(DEV, torch.bfloat16)
    router = torch.from_numpy(rng.normal(size=(32, 256)) / 16).to(DEV, torch.bfloat16)
    k = torch.from_numpy(rng.integers(1, 8, T).astype(np.int32)).to(DEV)
    d = B.LayerDesc(T=T, H=256, n_experts=8, n_sub=4, I_sub=64, k_max=7, score="sigmoid", renorm=True,
                    route_scale=1.5, expert_bias=torch.linspace(-0.5, 0.5, 8, device=DEV))
    st, ws = status(), torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    out = torch.full((T, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_layer_forward_quant(d, None, layer.packed, x, router, k, None, out, st, ws))
    idx = torch.empty(T, 7, dtype=torch.int32, device=DEV)
    tw = torch.empty(T, 7, dtype=torch.float32, device=DEV)
    B.check(B.moe_route(d, x, router, None, k, None, idx, tw, st, ws))
    assert B.moe_get_device_status(st) == 0
    x64, want, tol = to64(x), np.zeros((T, 256)), np.zeros((T, 256))
    for t in range(T):
        for j in range(int(k[t])):
            y, dy = layer.expert(int(idx[t, j]), x64[t:t + 1])
            g = float(tw[t, j])
            # the layer's own gates differ from the routing step's by the logits' errors, below 1e-4
            want[t] += g * y[0]
            tol[t] += g * (dy[0] + 1.5e-4 * np.abs(y[0]))
    within(out, want, tol + 2.0 ** -20 * np.abs(want))
