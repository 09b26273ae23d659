"""Products with packed 4-bit weights against float64: the projection, the grouped
experts, the shared expert and the whole layer.  Tolerances are sums of the
roundings that the float64 form counts (oracle/quant.py)."""
from dataclasses import replace

import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q
from quant_utils import DEV, Layer, pack, random_weights, status, to64, within

pytestmark = pytest.mark.gpu
KINDS = [("e2m1", 16), ("e2m1", 32), ("int4", 16), ("int4", 32)]


def _x(rng, T, K, ld=0):
    x = torch.full((T, max(ld, K)), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[:, :K] = torch.from_numpy(rng.normal(size=(T, K))).to(DEV, torch.bfloat16)
    return x


def _project(T, K, N, kind, group, swiglu, ldx=0, ldy=0, seed=0):
    rng = np.random.default_rng(seed + T + K + N)
    halves = 2 if swiglu else 1
    w = random_weights(rng, halves, N // halves, K, kind, group)
    x, out = _x(rng, T, K, ldx), N // halves
    d = B.QuantProject(T, K, N, kind, group, swiglu, ldx, ldy)
    y = torch.full((T, max(ldy, out)), 7.0, dtype=torch.bfloat16, device=DEV)
    ws, st = torch.empty(B.moe_quant_project_workspace_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_project(d, x, pack(w, kind, group), y, st, ws))
    assert B.moe_get_device_status(st) == 0
    assert (y[:, out:] == 7.0).all()
    w64, x64 = Q.weights(*w, kind, group), to64(x[:, :K])
    if swiglu:
        want = Q.swiglu(*Q.product(x64, w64[0]), *Q.product(x64, w64[1]))
    else:
        want = Q.product(x64, w64[0])
    within(y[:, :out], *want)


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T,K,N", [(1, 8, 1), (1, 1024, 256), (2, 136, 130), (5, 2056, 770), (8, 256, 129),
                                   (9, 512, 300), (16, 320, 64), (17, 264, 100), (33, 128, 128)])
def test_project_few_tokens(kind, group, T, K, N):
    _project(T, K, N, kind, group, False)


@pytest.mark.parametrize("kind,group", [("e2m1", 16), ("int4", 32)])
@pytest.mark.parametrize("T,K,N", [(64, 1024, 512), (100, 72, 33), (129, 640, 257), (300, 264, 130), (777, 128, 510),
                                   (1025, 8, 40)])
def test_project_many_tokens(kind, group, T, K, N):
    _project(T, K, N, kind, group, False)


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T,K,N", [(1, 7168, 512), (3, 264, 2), (8, 1000, 258), (20, 512, 600), (200, 264, 514)])
def test_project_swiglu(kind, group, T, K, N):
    _project(T, K, N, kind, group, True)


@pytest.mark.parametrize("T", [1, 6, 40, 300])
@pytest.mark.parametrize("swiglu", [False, True])
def test_project_strided_rows(T, swiglu):
    _project(T, 264, 130, "e2m1", 16, swiglu, ldx=272, ldy=143)


def _grouping(rng, T, E, k, skew=0.0):
    """(sorted_token, offsets) of k distinct experts for each token."""
    p = np.arange(1, E + 1.0) ** -skew
    unit = np.stack([rng.choice(E, size=k, replace=False, p=p / p.sum()) for _ in range(T)])
    order = np.argsort(unit.reshape(-1), kind="stable")
    offsets = np.concatenate(([0], np.cumsum(np.bincount(unit.reshape(-1), minlength=E))))
    return (order // k).astype(np.int32), offsets.astype(np.int32)


def _ffn(layer, T, k, seed=0, skew=0.0):
    rng = np.random.default_rng(seed)
    token, offsets = _grouping(rng, T, layer.E, k, skew)
    x = _x(rng, T, layer.H)
    d = B.LayerDesc(T=T, H=layer.H, n_experts=layer.E, n_sub=1, I_sub=layer.I, k_max=k)
    # the rows that no expert has stay as they were
    y = torch.full((T * k + 3, layer.H), 7.0, dtype=torch.bfloat16, device=DEV)
    st, ws = status(), torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    B.check(B.moe_grouped_ffn_quant(d, layer.packed, x, torch.from_numpy(token).to(DEV),
                                    torch.from_numpy(offsets).to(DEV), y, st, ws))
    assert B.moe_get_device_status(st) == 0
    assert (y[len(token):] == 7.0).all()
    x64 = to64(x)
    for e in range(layer.E):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            within(y[a:b], *layer.expert(e, x64[token[a:b]]), f"expert {e}")


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T,H,E,I,k", [(1, 64, 1, 64, 1), (5, 320, 8, 192, 3), (40, 256, 12, 128, 4), (150, 128, 3, 320, 2)])
def test_grouped_ffn(kind, group, T, H, E, I, k):  # noqa: E741
    _ffn(Layer(H + I, H, E, I, kind, group), T, k, seed=T)


@pytest.mark.parametrize("T,E,k,skew", [(700, 4, 1, 1.5), (400, 16, 5, 1.0), (64, 256, 2, 0.0)])
def test_grouped_ffn_ragged(T, E, k, skew):
    _ffn(Layer(E, 192, E, 64, "e2m1", 16), T, k, seed=T, skew=skew)


def _routed(d, x, router, k, ws, st, groups=None):
    """The selection that the layer makes, by the routing step alone."""
    d = replace(d, I_shared=0)
    idx = torch.empty(d.T, d.k_max, dtype=torch.int32, device=DEV)
    w = torch.empty(d.T, d.k_max, dtype=torch.float32, device=DEV)
    if groups is None:
        B.check(B.moe_route(d, x, router, None, k, None, idx, w, st, ws))
    else:
        B.check(B.moe_route_groups(d, groups, x, router, None, k, None, idx, w, None, None, st, ws))
    return idx.cpu().numpy(), to64(w)


def _layer(layer, T, k_max, seed=0, groups=None, score="softmax", renorm=False, scale=1.0, calls=1):
    rng = np.random.default_rng(seed)
    x = _x(rng, T, layer.H)
    router = torch.from_numpy(rng.normal(size=(layer.E, layer.H)) * layer.H ** -0.5).to(DEV, torch.bfloat16)
    k = torch.from_numpy(rng.integers(1, k_max + 1, T).astype(np.int32)).to(DEV)
    d = B.LayerDesc(T=T, H=layer.H, n_experts=layer.E, n_sub=1, I_sub=layer.I, k_max=k_max, score=score,
                    renorm=renorm, route_scale=scale, I_shared=layer.shared)
    ws, st = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV), status()
    out = torch.full((T, layer.H), float("nan"), dtype=torch.bfloat16, device=DEV)
    load = None if groups is None else torch.full((layer.E,), -1, dtype=torch.int32, device=DEV)
    for _ in range(calls):
        B.check(B.moe_layer_forward_quant(d, groups, layer.packed, x, router, k, load, out, st, ws))
    assert B.moe_get_device_status(st) == 0
    idx, w = _routed(d, x, router, k, ws, st, groups)
    x64 = to64(x)
    want, tol = np.zeros((T, layer.H)), np.zeros((T, layer.H))
    for t in range(T):
        for j in range(int(k[t])):
            y, dy = layer.expert(idx[t, j], x64[t:t + 1])
            # the gates of two computations of the logits: 2e-5 each (their own error) and the
            # logits', well below 1e-4
            want[t] += w[t, j] * y[0]
            # the activations may carry the gate, rounded with it
            tol[t] += np.abs(w[t, j]) * (dy[0] + 1.5e-4 * np.abs(y[0]))
    if layer.shared:
        y, dy = layer.shared_expert(x64)
        want, tol = want + y, tol + dy
    if groups is not None:
        assert load.cpu().numpy().tolist() == np.bincount(idx[idx >= 0], minlength=layer.E).tolist()
    within(out, want, tol + 2.0 ** -20 * np.abs(want))


@pytest.mark.parametrize("kind,group", KINDS)
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 40])
def test_layer(kind, group, T):
    _layer(Layer(T, 256, 16, 192, kind, group), T, 6, seed=T)


@pytest.mark.parametrize("T", [1, 4, 8, 12, 33])
def test_layer_grouped_and_shared(T):
    layer = Layer(T, 320, 32, 128, "e2m1", 16, shared=192)
    groups = B.GroupRoute(n_groups=8, groups_kept=4, group_best=2,
                          select_bias=torch.linspace(-0.02, 0.02, 32, device=DEV))
    _layer(layer, T, 4, seed=T, groups=groups, score="sigmoid", renorm=True, scale=2.5)


@pytest.mark.parametrize("T,H,E,I,k,shared", [(1, 2048, 256, 384, 16, 0), (3, 64, 1, 64, 1, 64), (8, 1024, 64, 64, 32, 0),
                                              (7, 192, 5, 704, 5, 320), (2, 4160, 4, 128, 2, 0)])
def test_layer_shapes(T, H, E, I, k, shared):  # noqa: E741
    _layer(Layer(H, H, E, I, "int4", 32, shared), T, k, seed=T, score="sigmoid", renorm=True, calls=3)


def test_shared_expert():
    for T in (1, 8, 70):
        layer = Layer(T, 256, 1, 64, "e2m1", 32, shared=192)
        rng = np.random.default_rng(T)
        x = _x(rng, T, 256)
        d = B.LayerDesc(T=T, H=256, n_experts=1, n_sub=1, I_sub=64, k_max=1, I_shared=192)
        ws, st = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV), status()
        y = torch.full((T, 256), 7.0, dtype=torch.bfloat16, device=DEV)
        B.check(B.moe_shared_ffn_quant(d, layer.packed, x, y, st, ws))
        assert B.moe_get_device_status(st) == 0
        within(y, *layer.shared_expert(to64(x)))
