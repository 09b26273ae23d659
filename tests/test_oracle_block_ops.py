"""Pins of the float64 forms of group routing, block norms and the adapter
projection: closed forms, brute force, and gradients against differences."""
import numpy as np
import pytest

from oracle import block_norm as N
from oracle import group_route as G
from oracle import lora as L


def test_routing_without_groups_is_a_plain_top_k():
    rng = np.random.default_rng(1)
    l = rng.standard_normal(24)
    u, w, _ = G.route_token(l, 5, "sigmoid", False, 1.0)
    assert u == list(np.argsort(-l, kind="stable")[:5])
    assert np.allclose(w, 1 / (1 + np.exp(-l[u])))


def test_bias_selects_but_does_not_weigh_and_groups_limit():
    # scores 0.5 everywhere: the bias alone decides, the weights stay equal
    bias = np.array([0.0, 0.3, 0.2, 0.0, 0.4, 0.0, 0.0, 0.1])
    u, w, _ = G.route_token(np.zeros(8), 3, "sigmoid", True, 2.0, bias=bias)
    assert u == [4, 1, 2] and np.allclose(w, 2 / 3)
    # groups {0,1},{2,3},{4,5},{6,7}: two best sums 1.3, 1.2, 1.4, 1.1; two groups stay
    u, _, _ = G.route_token(np.zeros(8), 3, "sigmoid", True, 2.0, 4, 2, 2, bias=bias)
    assert u == [4, 1, 0]
    # all equal: lower group, lower unit
    u, _, _ = G.route_token(np.zeros(8), 3, "softmax", False, 1.0, 4, 2, 1)
    assert u == [0, 1, 2]


def test_units_out_of_service():
    l = np.full(6, -np.inf)
    assert G.route_token(l, 3, "softmax", True, 1.0)[0] == []
    l[4] = 0.5
    u, w, _ = G.route_token(l, 3, "softmax", True, 1.0, 3, 1, 2)
    assert u == [4] and w == [1.0]
    assert G.route_token(np.array([np.nan, 1.0, np.inf]), 2, "sigmoid", False, 1.0)[0] == [1]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_routing_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    l, g = rng.standard_normal(12), rng.standard_normal(4)
    l[3] = -np.inf
    idx = [7, 2, 9, -1]

    def loss(v):
        s, _ = G.scores(v, score)
        w = s[idx[:3]]
        return 1.5 * (g[:3] * (w / w.sum() if renorm else w)).sum()

    d, _ = G.route_backward_token(l, idx, g, score, renorm, 1.5)
    for u in range(12):
        if u == 3:
            assert d[u] == 0
            continue
        h = np.zeros(12)
        h[u] = 1e-6
        assert abs((loss(l + h) - loss(l - h)) / 2e-6 - d[u]) < 1e-8


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_norm_gradients_against_differences(kind, post, pre):
    rng = np.random.default_rng(3)
    T, H = 3, 5
    shape = {"none": (1,), "channel": (H,), "token": (T,), "full": (T, H)}[kind]
    v = dict(r=rng.standard_normal((T, H)), y=rng.standard_normal((T, H)),
             gate=rng.standard_normal(shape), w_post=rng.standard_normal(H),
             w_pre=rng.standard_normal(H))
    d_out, d_h = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    kw = dict(offset=0.5, rs=0.9, bs=1.3, eps=1e-5)

    def loss(q):
        out, h, _ = N.forward(q["r"], q["y"], q["gate"], kind, q["w_post"] if post else None,
                              q["w_pre"] if pre else None, **kw)
        return (out * d_out).sum() + (0 if h is None else (h * d_h).sum())

    got = N.backward(v["r"], v["y"], v["gate"], kind, v["w_post"] if post else None,
                     v["w_pre"] if pre else None, d_out, d_h, **kw)
    names = {"d_residual": "r", "d_branch": "y", "d_gate": "gate", "d_w_post": "w_post",
             "d_w_pre": "w_pre"}
    assert set(got) == {"d_residual", "d_branch"} | ({"d_gate"} if kind != "none" else set()) | (
        {"d_w_post"} if post else set()) | ({"d_w_pre"} if pre else set())
    for name, (g, size) in got.items():
        assert (np.abs(g) <= size + 1e-12).all()
        for at in np.ndindex(g.shape):
            up = {k: x.copy() for k, x in v.items()}
            dn = {k: x.copy() for k, x in v.items()}
            up[names[name]][at] += 1e-6
            dn[names[name]][at] -= 1e-6
            assert abs((loss(up) - loss(dn)) / 2e-6 - g[at]) < 1e-7


def test_norm_of_a_constant_row():
    out, h, _ = N.forward(np.full((1, 4), 3.0), w_pre=np.ones(4), eps=0.0)
    assert (out == 3.0).all() and np.allclose(h, 1.0)


def test_adapter_projection_equals_merged_weights():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((6, 8)), rng.standard_normal((10, 8))
    a, b = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 10, 3))
    a[:, 2:] = np.nan                      # past the ranks
    b[:, :, 2:] = np.nan
    adapter = np.array([0, 1, -1, 1, 0, 0])
    y, _, _ = L.project(x, w, a, b, [2, 1], [0.5, 2.0], adapter)
    for t, i in enumerate(adapter):
        m = w if i < 0 else w + [0.5, 2.0][i] * b[i][:, :[2, 1][i]] @ a[i, :[2, 1][i]]
        assert np.allclose(y[t], m @ x[t])
    z, _, _ = L.project(x, w, a, b, [2, 1], [0.5, 2.0], adapter, swiglu=True)
    assert np.allclose(z, y[:, :5] / (1 + np.exp(-y[:, :5])) * y[:, 5:])
