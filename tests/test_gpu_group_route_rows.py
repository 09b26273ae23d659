"""The gradient of routing, and routing itself, over more tokens than a launch has
warps for at once."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _many():
    """Above the tokens of one turn of any routing kernel: 8 CTAs of 8 warps a SM."""
    return 64 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("E,k", [(128, 8), (256, 8), (60, 5), (250, 3), (16, 16)])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                          ("sigmoid", True)])
def test_gradient_of_many_tokens(E, k, score, renorm):
    """Against the formula in float64: 2e-5 of the size of its terms, as for few tokens."""
    T = 2 * _many() + 777
    g = torch.Generator(device=DEV).manual_seed(E + k)
    l = torch.randn(T, E, generator=g, device=DEV)
    l[torch.rand(T, E, generator=g, device=DEV) < 0.03] = float("-inf")
    idx = torch.argsort(torch.rand(T, E, generator=g, device=DEV), dim=1)[:, :k].to(torch.int32)
    idx[torch.rand(T, k, generator=g, device=DEV) < 0.1] = -1
    dw = torch.randn(T, k, generator=g, device=DEV)
    d = B.LayerDesc(T=T, H=64, n_experts=E, n_sub=1, I_sub=64, k_max=k, score=score, renorm=renorm,
                    route_scale=2.5)
    got = torch.full((T, E), 99.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.check(B.moe_route_backward(d, l, idx, dw, got, st))
    assert B.moe_get_device_status(st) == 0
    l64, live = l.double(), idx >= 0
    at = idx.clamp(min=0).long()
    live &= torch.gather(l, 1, at) > float("-inf")
    gw = torch.where(live, 2.5 * dw.double(), 0.0)

    def rows(v):
        return torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(1, at, torch.where(live, v, 0.0))

    if score == "softmax" and not renorm:
        s, ds = torch.nan_to_num(torch.softmax(l64, 1)), rows(gw)
        ref = s * (ds - (ds * s).sum(1, keepdim=True))
        size = s * (ds.abs() + (ds.abs() * s).sum(1, keepdim=True))
    else:
        sel = torch.where(live, torch.gather(l64, 1, at), float("-inf"))
        if score == "softmax":
            w, f = torch.nan_to_num(torch.softmax(sel, 1)), torch.ones_like(sel)
        else:
            w, f = torch.sigmoid(sel), 1 - torch.sigmoid(sel)
            if renorm:
                w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        dot, dots = (gw * w).sum(1, keepdim=True), (gw.abs() * w).sum(1, keepdim=True)
        if not renorm:
            dot, dots = 0 * dot, 0 * dots
        ref, size = rows(w * f * (gw - dot)), rows(w * f * (gw.abs() + dots))
    assert ((got.double() - ref).abs() <= 2e-5 * size + 1e-30).all()


@pytest.mark.parametrize("E,groups,kept,k", [(256, 8, 4, 8), (128, 1, 1, 16), (128, 64, 20, 8), (60, 1, 1, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_of_every_turn_are_routed_alike(E, groups, kept, k, score):
    """Each token of a long call as in a call of its own turn, and the loads of all."""
    part = 500
    T = 5 * part * ((_many() + part - 1) // part)
    g = torch.Generator(device=DEV).manual_seed(E + groups)
    one = torch.randn(part, E, generator=g, device=DEV)
    one[torch.rand(part, E, generator=g, device=DEV) < 0.05] = float("-inf")
    kt = torch.randint(1, k + 1, (part,), generator=g, device=DEV, dtype=torch.int32)
    bias = 0.05 * torch.randn(E, generator=g, device=DEV)

    def run(l, kt):
        T = l.shape[0]
        d = B.LayerDesc(T=T, H=64, n_experts=E, n_sub=1, I_sub=64, k_max=k, score=score, renorm=True,
                        route_scale=2.5)
        new = lambda *s, dtype=torch.int32: torch.full(s, -7, dtype=dtype, device=DEV)  # noqa: E731
        idx, w, k_out, load, st = new(T, k), new(T, k, dtype=torch.float32), new(T), new(E), torch.zeros(
            1, dtype=torch.int32, device=DEV)
        B.check(B.moe_route_groups(d, B.GroupRoute(groups, kept, 1, bias), None, None, l, kt, None, idx, w,
                                   k_out, load, st, None))
        assert B.moe_get_device_status(st) == 0
        return idx, w, k_out, load

    few = run(one, kt)
    n = T // part
    many = run(one.repeat(n, 1), kt.repeat(n))
    for a, b in zip(few[:3], many[:3]):
        assert torch.equal(a.repeat(n, *([1] * (a.dim() - 1))), b)
    assert torch.equal(few[3] * n, many[3])
    idx = few[0].cpu().numpy()
    assert (np.bincount(idx[idx >= 0], minlength=E) == few[3].cpu().numpy()).all()
