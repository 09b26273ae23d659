"""moe_route_groups, moe_route_backward and the layer built on them against
the float64 forms.

Selection: where no decision of a token hangs on less than 2e-6 of its largest
value (the fp32 scores are within 1e-6), units and order are equal; equal
scores are exact ties on both sides.  Weights: expf (2 ulp), a division and a
sum of at most E terms: (E + 16) 2^-24 relative, plus the smallest normal.
Gradients: the same relative error of every term, so 2e-5 of the sum of their
sizes.
"""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import group_route as G

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _desc(T, E, k, score="sigmoid", renorm=True, **kw):
    return B.LayerDesc(T=T, H=64, n_experts=E, n_sub=1, I_sub=64, k_max=k, score=score,
                       renorm=renorm, route_scale=2.5, **kw)


def _inputs(T, E, k, seed, masked=0.0):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < masked] = -np.inf
    bias = (rng.integers(-20, 21, E) * 0.001).astype(np.float32)
    kt = rng.integers(1, k + 1, T).astype(np.int32)
    return l, bias, kt


def _run(l, bias, kt, k, groups, kept, best, score, renorm, with_load=True):
    T, E = l.shape
    d = _desc(T, E, k, score, renorm)
    g = B.GroupRoute(groups, kept, best, None if bias is None else torch.tensor(bias, device=DEV))
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    k_out = torch.full((T,), -7, dtype=torch.int32, device=DEV)
    load = torch.full((E,), -7, dtype=torch.int32, device=DEV) if with_load else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_groups(d, g, None, None, torch.tensor(l, device=DEV),
                               torch.tensor(kt, device=DEV), None, idx, w, k_out, load, st, None))
    return (idx.cpu().numpy(), w.cpu().numpy(), k_out.cpu().numpy(),
            load.cpu().numpy() if with_load else None, B.moe_get_device_status(st))


def _check(l, bias, kt, k, groups, kept, best, score, renorm, status=0):
    T, E = l.shape
    idx, w, k_out, load, st = _run(l, bias, kt, k, groups, kept, best, score, renorm)
    assert st == status
    unsure = 0
    for t in range(T):
        u, ref, gap = G.route_token(l[t], int(kt[t]), score, renorm, 2.5, groups, kept, best, bias)
        n = len(u)
        assert k_out[t] == n
        assert (idx[t, n:] == -1).all() and (w[t, n:] == 0).all()
        biggest = G.scores(l[t], score)[0].max()
        if bias is not None:
            biggest += np.abs(bias[np.isfinite(bias)]).max()
        if gap < 2e-6 * biggest:
            unsure += 1
            continue
        assert list(idx[t, :n]) == u, t
        assert (np.abs(w[t, :n] - ref) <= (E + 16) * 2.0 ** -24 * np.abs(ref) + 1e-37).all()
    assert unsure <= max(1, T // 50)
    assert (load == np.bincount(idx[idx >= 0], minlength=E)).all()


SHAPES = [  # E, groups, kept, best, k
    (256, 8, 4, 2, 8), (256, 8, 3, 1, 8), (128, 1, 1, 1, 16), (256, 1, 1, 1, 32), (160, 8, 3, 2, 6),
    (132, 4, 2, 2, 9), (64, 64, 20, 1, 8), (256, 128, 11, 2, 8), (195, 65, 7, 2, 12), (60, 1, 1, 2, 4),
    (8, 2, 1, 2, 3), (1, 1, 1, 1, 1), (33, 3, 2, 2, 5), (255, 17, 5, 2, 8), (231, 33, 4, 2, 8),
    (32, 32, 9, 1, 9), (256, 256, 40, 1, 8), (64, 4, 4, 2, 8), (96, 16, 4, 2, 4),
]


@pytest.mark.parametrize("E,groups,kept,best,k", SHAPES)
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", False)])
def test_selection_and_weights(E, groups, kept, best, k, score, renorm):
    l, bias, kt = _inputs(131, E, k, E * 1000 + groups)
    _check(l, bias, kt, k, groups, kept, best, score, renorm)


@pytest.mark.parametrize("T", [1, 2, 8, 9, 2500])
@pytest.mark.parametrize("score,renorm", [("sigmoid", False), ("softmax", True)])
def test_token_counts(T, score, renorm):
    l, bias, kt = _inputs(T, 64, 6, T)
    _check(l, bias, kt, 6, 8, 3, 2, score, renorm)


def test_more_tokens_than_resident_warps():
    l, bias, kt = _inputs(6000, 32, 4, 5)
    _check(l, bias, kt, 4, 4, 2, 2, "sigmoid", True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept", [(8, 4), (1, 1), (64, 30)])
def test_units_out_of_service(score, groups, kept):
    l, bias, kt = _inputs(200, 64, 8, 11, masked=0.8)
    l[3] = -np.inf                    # nothing left
    l[4] = -np.inf
    l[4, 63] = 0.25                   # one unit left
    _check(l, bias, kt, 8, groups, kept, 2, score, True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_group_and_unit(score):
    rng = np.random.default_rng(3)
    l = rng.choice(np.array([-1.5, -0.0, 0.0, 0.25, 2.0], dtype=np.float32), size=(100, 64))
    l[0] = 0.5
    kt = np.full(100, 8, dtype=np.int32)
    # softmax: equal logits give equal scores, and no sum of two differs in rounding
    for groups, kept, best in ((8, 3, 1), (8, 3, 2), (1, 1, 1), (64, 9, 1)):
        _check(l, None, kt, 8, groups, kept, best, score, True)


def test_saturated_and_extreme_logits():
    l = np.array([[200.0, -200.0, 88.0, -88.0, 0.0, 1e30, -1e30, 3.0]], dtype=np.float32)
    idx, w, _, _, st = _run(l, None, np.array([8], np.int32), 8, 1, 1, 1, "sigmoid", False)
    assert st == 0 and np.isfinite(w).all()
    # 200 and 1e30 both score 1: the lower unit first
    assert list(idx[0, :3]) == [0, 2, 5] and (w[0, :3] == 2.5).all()
    idx, w, _, _, st = _run(l, None, np.array([8], np.int32), 8, 1, 1, 1, "softmax", True)
    assert st == 0 and idx[0, 0] == 5 and w[0, 0] == 2.5 and np.isfinite(w).all()


def test_all_selected_scores_zero():
    l = np.full((2, 8), -500.0, dtype=np.float32)
    _, w, k_out, _, st = _run(l, None, np.array([3, 8], np.int32), 8, 2, 2, 1, "sigmoid", True)
    assert st == 0 and list(k_out) == [3, 8]        # equal weights of the underflown scores
    assert np.allclose(w[0, :3], 2.5 / 3) and np.allclose(w[1], 2.5 / 8)
    _, w, _, _, _ = _run(l, None, np.array([3, 8], np.int32), 8, 2, 2, 1, "sigmoid", False)
    assert (w == 0).all()
    _, w, _, _, _ = _run(l, None, np.array([4, 4], np.int32), 4, 1, 1, 1, "softmax", True)
    assert np.allclose(w, 2.5 / 4)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_non_finite_logits_leave_and_are_reported(value, score):
    l, bias, kt = _inputs(40, 64, 8, 21)
    l[7, 13] = value
    l[9, :] = value
    _check(l, bias, kt, 8, 8, 4, 2, score, True, status=6)


def test_bias_takes_units_out_and_nan_is_reported():
    l, bias, kt = _inputs(64, 64, 8, 22)
    bias[5] = -np.inf
    _check(l, bias, kt, 8, 8, 4, 2, "sigmoid", True)
    bias[9] = np.nan
    idx, _, _, _, st = _run(l, bias, kt, 8, 8, 4, 2, "sigmoid", True)
    assert st == 6 and not (idx == 9).any() and not (idx == 5).any()


def test_budgets_out_of_range_are_reported_and_clamped():
    l, bias, _ = _inputs(4, 64, 8, 23)
    _, _, k_out, _, st = _run(l, bias, np.array([0, 9, -3, 5], np.int32), 8, 8, 4, 2, "sigmoid", True)
    assert st == 7 and list(k_out) == [0, 8, 0, 5]


def test_without_bias_or_load():
    l, _, kt = _inputs(64, 64, 8, 24)
    assert _run(l, None, kt, 8, 8, 4, 2, "sigmoid", True, with_load=False)[4] == 0
    _check(l, None, kt, 8, 8, 4, 2, "sigmoid", True)


@pytest.mark.parametrize("T", [1, 40, 200])
@pytest.mark.parametrize("E,groups", [(64, 8), (60, 4)])
def test_from_x_and_router_weights(T, E, groups):
    """Logits computed inside (CUDA cores and tensor cores): the selection on
    the logits that come out."""
    g = torch.Generator(device=DEV).manual_seed(T)
    H, k = 256, 6
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    rw = (torch.randn(E, H, generator=g, device=DEV) / 16).bfloat16()
    eb = torch.randn(E, generator=g, device=DEV)
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=64, k_max=k, score="sigmoid", renorm=True,
                    route_scale=2.5, expert_bias=eb)
    gr = B.GroupRoute(groups, 2, 2)
    lo = torch.empty(T, E, device=DEV)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.moe_workspace_size(d), dtype=torch.uint8, device=DEV)
    kt = torch.full((T,), k, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_groups(d, gr, x, rw, None, kt, lo, idx, w, None, None, st, ws))
    assert B.moe_get_device_status(st) == 0
    ref = x.double() @ rw.double().t() + eb.double()
    bound = H * 2.0 ** -24 * (x.double().abs() @ rw.double().abs().t()) + 1e-6
    assert ((lo.double() - ref).abs() <= bound).all()
    l = lo.cpu().numpy()
    for t in range(T):
        u, rw_, gap = G.route_token(l[t], k, "sigmoid", True, 2.5, groups, 2, 2)
        if gap > 2e-6:
            assert list(idx[t].cpu().numpy()) == u


@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (60, 5), (1, 1), (33, 32)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward(E, k, score, renorm):
    T = 150
    rng = np.random.default_rng(E + k)
    l, _, kt = _inputs(T, E, k, E, masked=0.1 if E > 8 else 0.0)
    if E > 8:
        l[5] = -np.inf
    l[6] -= 300.0
    idx = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        idx[t, :kt[t]] = rng.choice(E, kt[t], replace=False)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    _check_backward(l, idx, dw, k, score, renorm)


def _check_backward(l, idx, dw, k, score, renorm, status=0):
    T, E = l.shape
    out = torch.full((T, E), 7.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_backward(_desc(T, E, k, score, renorm), torch.tensor(l, device=DEV),
                                 torch.tensor(idx, device=DEV), torch.tensor(dw, device=DEV), out, st))
    assert B.moe_get_device_status(st) == status
    got = out.cpu().numpy()
    for t in range(T):
        ref, size = G.route_backward_token(l[t], idx[t], dw[t], score, renorm, 2.5)
        assert (np.abs(got[t] - ref) <= 2e-5 * size + 1e-37).all(), t


def test_backward_gradient_follows_the_forward_weights():
    """Differences of the float64 forward form at the GPU's own selection."""
    l, bias, kt = _inputs(6, 64, 8, 31)
    idx = _run(l, bias, kt, 8, 8, 4, 2, "sigmoid", True)[0]
    dw = np.random.default_rng(0).standard_normal((6, 8)).astype(np.float32)
    out = torch.empty(6, 64, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_backward(_desc(6, 64, 8), torch.tensor(l, device=DEV),
                                 torch.tensor(idx, device=DEV), torch.tensor(dw, device=DEV), out, st))
    got = out.cpu().numpy()

    def loss(v, t):
        u = idx[t][idx[t] >= 0]
        s = 1 / (1 + np.exp(-v[u]))
        return 2.5 * (dw[t, :len(u)] * s / s.sum()).sum()

    for t in range(6):
        for u in list(idx[t][idx[t] >= 0]) + [0, 63]:
            h = np.zeros(64)
            h[u] = 1e-5
            v = l[t].astype(np.float64)
            assert abs((loss(v + h, t) - loss(v - h, t)) / 2e-5 - got[t, u]) < 1e-5


def test_backward_reports_bad_units():
    l, _, _ = _inputs(3, 64, 4, 41)
    idx = np.array([[1, 2, 3, 4], [5, 64, 6, -1], [7, 9, 7, -1]], dtype=np.int32)
    dw = np.ones((3, 4), dtype=np.float32)
    out = torch.empty(3, 64, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_backward(_desc(3, 64, 4, "sigmoid", False), torch.tensor(l, device=DEV),
                                 torch.tensor(idx, device=DEV), torch.tensor(dw, device=DEV), out, st))
    assert B.moe_get_device_status(st) == 8
    clean = np.array([[1, 2, 3, 4], [5, -1, 6, -1], [7, 9, -1, -1]], dtype=np.int32)
    got = out.cpu().numpy()
    for t in range(3):
        ref, size = G.route_backward_token(l[t], clean[t], dw[t], "sigmoid", False, 2.5)
        assert (np.abs(got[t] - ref) <= 2e-5 * size + 1e-37).all()


def test_backward_masked_softmax_with_nan():
    l, _, kt = _inputs(20, 64, 4, 42)
    l[2, 5] = np.nan
    idx = np.tile(np.array([5, 6, 7, -1], np.int32), (20, 1))
    dw = np.ones((20, 4), dtype=np.float32)
    _check_backward(l, idx, dw, 4, "softmax", False, status=6)


@pytest.mark.parametrize("T", [3, 200])
def test_layer_matches_its_component_calls(T):
    from aware_moe_expert_gb300 import inputs
    from aware_moe_expert_gb300.workloads import TINY
    wl = TINY.with_T(T)
    d_in = inputs.make_layer_inputs(wl, DEV)
    d = B.desc_for(wl, expert_bias=d_in["expert_bias"])
    bias = torch.linspace(-0.02, 0.02, wl.E_r, device=DEV)
    g = B.GroupRoute(wl.n_experts, 6, 2, bias)
    ws = torch.empty(B.moe_workspace_size(d), dtype=torch.uint8, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kt = d_in["k_per_token"]
    out = torch.empty(T, wl.H, dtype=torch.bfloat16, device=DEV)
    load = torch.empty(wl.E_r, dtype=torch.int32, device=DEV)
    B.check(B.moe_layer_forward_groups(d, g, d_in["x"], d_in["router_w"], d_in["w_gate_up"],
                                       d_in["w_down"], kt, load, out, st, ws))
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    n = T * wl.k_max
    idx, w, ko = i32(T, wl.k_max), torch.empty(T, wl.k_max, device=DEV), i32(T)
    load2 = i32(wl.E_r)
    B.check(B.moe_route_groups(d, g, d_in["x"], d_in["router_w"], None, kt, None, idx, w, ko, load2,
                               st, ws))
    counts, offsets, srt, inv = i32(wl.E_r), i32(wl.E_r + 1), i32(n), i32(n)
    B.check(B.moe_permute(d, idx, ko, counts, offsets, srt, inv, st, ws))
    y = torch.empty(n, wl.H, dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_grouped_ffn(d, d_in["x"], srt, offsets, d_in["w_gate_up"], d_in["w_down"], y, st, ws))
    out2 = torch.empty_like(out)
    B.check(B.moe_combine(d, y, None, inv, w, ko, out2, st))
    assert B.moe_get_device_status(st) == 0
    assert torch.equal(out, out2) and torch.equal(load, load2) and torch.equal(load, counts)


def test_repeats_to_the_bit_on_another_stream():
    l, bias, kt = _inputs(3000, 256, 8, 51)
    a = _run(l, bias, kt, 8, 8, 4, 2, "sigmoid", True)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = _run(l, bias, kt, 8, 8, 4, 2, "sigmoid", True)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)
