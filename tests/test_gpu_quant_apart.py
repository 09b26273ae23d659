"""4-bit calls that have to stay apart: tokens that are not finite in a layer, and calls that
run at once, captured or not, each with its own workspace."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from quant_utils import DEV, Layer, pack, random_weights, status

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _bf(rng, *shape):
    return torch.from_numpy(rng.normal(size=shape)).to(DEV, torch.bfloat16)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [3, 4, 7, 8, 16, 90])
def test_a_token_of_a_layer_that_is_not_finite(T, bad):
    """Routing reports it; the others' bits are those of a call without it."""
    layer = Layer(T, 256, 16, 128, "int4", 32, shared=64)
    rng = np.random.default_rng(T)
    router, x = _bf(rng, 16, 256) * 256 ** -0.5, _bf(rng, T, 256)
    k = torch.from_numpy(rng.integers(1, 5, T).astype(np.int32)).to(DEV)
    d = B.LayerDesc(T=T, H=256, n_experts=16, n_sub=1, I_sub=128, k_max=4, score="sigmoid", renorm=True, I_shared=64)
    for groups in (None, B.GroupRoute(n_groups=4, groups_kept=2, select_bias=torch.zeros(16, device=DEV))):
        outs = []
        for broken in (False, True):
            if broken:
                x = x.clone()
                x[1, 100] = bad
            st, out = status(), torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
            ws = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
            B.check(B.moe_layer_forward_quant(d, groups, layer.packed, x, router, k, None, out, st, ws))
            assert B.moe_get_device_status(st) == (6 if broken else 0)
            outs.append(out)
        x = x.clone()
        x[1, 100] = 0.5
        rest = [t for t in range(T) if t != 1]
        assert torch.equal(outs[0][rest], outs[1][rest])


def _project(rng, T, K, N, kind, group, swiglu):
    halves = 2 if swiglu else 1
    d = B.QuantProject(T, K, N, kind, group, swiglu)
    w, x = pack(random_weights(rng, halves, N // halves, K, kind, group), kind, group), _bf(rng, T, K)
    y, st = torch.full((T, N // halves), 7.0, dtype=torch.bfloat16, device=DEV), status()
    ws = torch.empty(B.moe_quant_project_workspace_size(d), dtype=torch.uint8, device=DEV)

    def run(stream=None):
        B.check(B.moe_quant_project(d, x, w, y, st, ws, stream))
    return run, y, st


@pytest.mark.parametrize("T,K,N,swiglu", [(1, 7168, 512, False), (8, 1000, 258, True), (40, 2056, 770, False),
                                          (64, 1024, 1024, True), (700, 264, 514, False)])
def test_captured_projections_at_once(T, K, N, swiglu):
    """Two graphs of several calls each on two streams, over and over, and calls between them."""
    rng = np.random.default_rng(T)
    calls = [_project(rng, T, K, N, *kind, swiglu) for kind in (("e2m1", 16), ("int4", 32))]
    want, graphs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    for run, y, _ in calls:
        run()
        want.append(y.clone())
    torch.cuda.synchronize()
    for (run, y, _), s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                run()
        y.fill_(7.0)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s, (run, _, _) in zip(graphs, streams, calls):
            with torch.cuda.stream(s):
                g.replay()
            run(s)
    torch.cuda.synchronize()
    for (_, y, st), w in zip(calls, want):
        assert torch.equal(y, w) and B.moe_get_device_status(st) == 0


@pytest.mark.parametrize("T", [2, 8, 50])
def test_steps_of_a_layer_at_once(T):
    """The shared expert on one stream, the routed ones on another, a workspace each."""
    layer = Layer(T, 320, 8, 192, "e2m1", 16, shared=256)
    rng = np.random.default_rng(T)
    x = _bf(rng, T, 320)
    unit = np.stack([rng.choice(8, size=3, replace=False) for _ in range(T)]).reshape(-1)
    order = np.argsort(unit, kind="stable")
    token = torch.from_numpy((order // 3).astype(np.int32)).to(DEV)
    offsets = torch.from_numpy(np.concatenate(([0], np.cumsum(np.bincount(unit, minlength=8)))).astype(np.int32)).to(DEV)
    d = B.LayerDesc(T=T, H=320, n_experts=8, n_sub=1, I_sub=192, k_max=3, I_shared=256)
    ws = [torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    st, y = status(), torch.empty(T * 3, 320, dtype=torch.bfloat16, device=DEV)
    ysh = torch.empty(T, 320, dtype=torch.bfloat16, device=DEV)

    def routed(s=None):
        B.check(B.moe_grouped_ffn_quant(d, layer.packed, x, token, offsets, y, st, ws[0], s))

    def shared(s=None):
        B.check(B.moe_shared_ffn_quant(d, layer.packed, x, ysh, st, ws[1], s))
    routed()
    shared()
    torch.cuda.synchronize()
    want = y.clone(), ysh.clone()
    y.fill_(7.0)
    ysh.fill_(7.0)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        routed(a)
        shared(b)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(ysh, want[1]) and B.moe_get_device_status(st) == 0
