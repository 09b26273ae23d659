"""moe_block_norm and its backward pass against the float64 forms.

fp32 outputs: every value is a few roundings of its terms and a mean of H
squares summed in fp32 (at most 16 terms in a thread, then a tree): 2e-6 of the
terms' size, times 8 for the products the chain multiplies.  bf16 outputs add
half an ulp (2^-8 of the value).  Column sums add T terms in fp32, in chains of
at most T / CTAs + 32: 2e-5 of the terms' size.
"""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import block_norm as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
REL = 1.6e-5


def _bf(t):
    return 2.0 ** -8 if t == BF16 else 0.0


def _make(T, H, res, act, kind, seed, ld=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rows(dtype, std):
        width = ld or H
        return (torch.randn(T, width, generator=g, device=DEV) * std).to(dtype)[:, :H]

    shape = {"channel": (H,), "token": (T,)}.get(kind)
    v = dict(r=rows(res, 2.0 * scale), y=rows(act, 0.7 * scale))
    v["gate"] = None if kind == "none" else rows(act, 0.5) if kind == "full" else (
        torch.randn(shape, generator=g, device=DEV) * 0.5).to(act)
    v["w_post"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(act)
    v["w_pre"] = (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(act)
    v["d_out"], v["d_h"] = rows(res, 1.0), rows(act, 1.0)
    return v


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _desc(v, T, H, res, act, kind, post, pre, ld=0, **kw):
    return B.BlockNormDesc(T=T, H=H, residual_dtype=res, act_dtype=act, gate=kind,
                           w_post=v["w_post"] if post else None, w_pre=v["w_pre"] if pre else None,
                           ld_residual=ld, ld_branch=ld, ld_gate=ld, ld_out=ld, ld_normed=ld,
                           eps=1e-5, weight_offset=0.25, residual_scale=0.9, branch_scale=1.25,
                           **kw)


KW = dict(offset=0.25, rs=0.9, bs=1.25, eps=1e-5)


def _out(v, ld, dtype):
    T, H = v["r"].shape
    return torch.full((T, ld or H), 99.0, device=DEV, dtype=dtype)[:, :H]


def _forward(T, H, res, act, kind, post, pre, ld=0, branch=True, seed=0, scale=1.0):
    v = _make(T, H, res, act, kind, seed + T * 7 + H, ld, scale)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = _desc(v, T, H, res, act, kind, post, pre, ld, dev_status=st)
    out = _out(v, ld, res)
    h = _out(v, ld, act) if pre else None
    B.check(B.moe_block_norm(d, v["r"], v["y"] if branch else None, v["gate"], out, h))
    assert B.moe_get_device_status(st) == 0
    ref, ref_h, mag = N.forward(_np(v["r"]), _np(v["y"]) if branch else None, _np(v["gate"]), kind,
                                _np(v["w_post"]) if post else None, _np(v["w_pre"]) if pre else None,
                                **KW)
    assert (np.abs(_np(out) - ref) <= _bf(res) * np.abs(ref) + REL * mag).all()
    if pre:
        f = 1 / np.sqrt((ref * ref).mean(1, keepdims=True) + 1e-5)
        size = mag * f * np.abs(_np(v["w_pre"]) + 0.25)
        assert (np.abs(_np(h) - ref_h) <= _bf(act) * np.abs(ref_h) + REL * (size + np.abs(ref_h))).all()
    return v, out, h


TYPES = [(BF16, BF16), (F32, BF16), (F32, F32)]


@pytest.mark.parametrize("res,act", TYPES)
@pytest.mark.parametrize("H", [1, 7, 8, 31, 64, 250, 256, 1001, 2048, 4104])
def test_forward_sizes(H, res, act):
    _forward(37, H, res, act, "none", True, True)


@pytest.mark.parametrize("res,act", TYPES)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("H", [96, 101])
def test_forward_kinds(H, post, pre, kind, res, act):
    _forward(50, H, res, act, kind, post, pre)


@pytest.mark.parametrize("T", [1, 2, 151, 152, 153, 1300])
def test_forward_tokens(T):
    _forward(T, 256, BF16, BF16, "full", True, True)


@pytest.mark.parametrize("H,res,act", [(7168, BF16, BF16), (8192, F32, F32), (8200, BF16, BF16),
                                       (16384, F32, F32), (16383, BF16, BF16), (12289, F32, BF16)])
def test_forward_wide(H, res, act):
    _forward(5, H, res, act, "channel", True, True)


@pytest.mark.parametrize("H,ld", [(64, 72), (64, 67), (33, 40), (2048, 4096)])
def test_forward_strided_rows(H, ld):
    _, out, h = _forward(23, H, BF16, BF16, "full", True, True, ld=ld)
    for t in (out, h):     # nothing between the rows is written
        base = torch.as_strided(t, (23, ld), (ld, 1))
        assert (base[:22, H:] == 99).all()


def test_forward_without_branch_and_pre_norm_only():
    _forward(19, 128, BF16, BF16, "none", False, True, branch=False)
    v = _make(19, 128, BF16, BF16, "none", 3)
    d = _desc(v, 19, 128, BF16, BF16, "none", False, True)
    h = torch.empty(19, 128, dtype=BF16, device=DEV)
    B.check(B.moe_block_norm(d, v["r"], None, None, None, h))
    ref = N.forward(_np(v["r"]), w_pre=_np(v["w_pre"]), **KW)[1]
    assert (np.abs(_np(h) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * REL * np.abs(ref)).all()


def test_forward_in_place_and_misaligned_start():
    v = _make(300, 512, BF16, BF16, "none", 5)
    d = _desc(v, 300, 512, BF16, BF16, "none", True, True)
    a, h = torch.empty_like(v["r"]), torch.empty_like(v["r"])
    B.check(B.moe_block_norm(d, v["r"], v["y"], None, a, h))
    b, h2 = v["r"].clone(), torch.empty_like(h)
    B.check(B.moe_block_norm(d, b, v["y"], None, b, h2))
    assert torch.equal(a, b) and torch.equal(h, h2)
    # the same rows one element off the 16-byte grid
    buf = torch.zeros(300 * 512 + 8, dtype=BF16, device=DEV)
    r = buf[1:1 + 300 * 512].view(300, 512)
    r.copy_(v["r"])
    c = torch.empty_like(a)
    B.check(B.moe_block_norm(d, r, v["y"], None, c, h2))
    # another order of the row sums: half an ulp on either side
    assert ((a.float() - c.float()).abs() <= 2.0 ** -7 * a.float().abs() + 1e-6).all()


def test_zero_rows_and_zero_tokens():
    v = _make(4, 64, BF16, BF16, "none", 6)
    v["r"].zero_()
    v["y"].zero_()
    d = _desc(v, 4, 64, BF16, BF16, "none", True, True)
    out, h = torch.empty_like(v["r"]), torch.empty_like(v["r"])
    B.check(B.moe_block_norm(d, v["r"], v["y"], None, out, h))
    assert (out == 0).all() and (h == 0).all()
    d0 = _desc(v, 0, 64, BF16, BF16, "channel", True, True)
    dw = [torch.full((64,), 5.0, device=DEV) for _ in range(3)]
    ws = torch.empty(max(1, B.moe_block_norm_workspace_size(d0)), dtype=torch.uint8, device=DEV)
    B.check(B.moe_block_norm_backward(d0, None, None, None, None, None, None, None, dw[0], dw[1],
                                      dw[2], ws))
    assert all((w == 0).all() for w in dw)


def test_a_row_of_nan_stays_in_its_row():
    v = _make(40, 64, BF16, BF16, "none", 8)
    v["y"][7, 3] = float("nan")
    v["r"][9, 5] = float("inf")
    d = _desc(v, 40, 64, BF16, BF16, "none", True, True)
    out, h = torch.empty_like(v["r"]), torch.empty_like(v["r"])
    B.check(B.moe_block_norm(d, v["r"], v["y"], None, out, h))
    rows = [t for t in range(40) if t not in (7, 9)]
    assert torch.isfinite(out[rows].float()).all() and torch.isfinite(h[rows].float()).all()
    assert out[7].isnan().all() and out[9, 5].isinf()


def _backward(T, H, res, act, kind, post, pre, ld=0, branch=True, with_out=True, seed=0):
    v = _make(T, H, res, act, kind, seed + T * 11 + H, ld)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = _desc(v, T, H, res, act, kind, post, pre, ld, dev_status=st)
    ws = torch.empty(B.moe_block_norm_workspace_size(d), dtype=torch.uint8, device=DEV)
    got = {"d_residual": _out(v, ld, res)}
    if branch:
        got["d_branch"] = _out(v, ld, act)
    if kind != "none":
        got["d_gate"] = _out(v, ld, act) if kind == "full" else torch.full(
            (H if kind == "channel" else T,), 99.0, device=DEV)
    if post:
        got["d_w_post"] = torch.full((H,), 99.0, device=DEV)
    if pre:
        got["d_w_pre"] = torch.full((H,), 99.0, device=DEV)

    def call():
        B.check(B.moe_block_norm_backward(
            d, v["r"], v["y"] if branch else None, v["gate"], v["d_out"] if with_out else None,
            v["d_h"] if pre else None, got["d_residual"], got.get("d_branch"), got.get("d_gate"),
            got.get("d_w_post"), got.get("d_w_pre"), ws))

    call()
    assert B.moe_get_device_status(st) == 0
    ref = N.backward(_np(v["r"]), _np(v["y"]) if branch else None, _np(v["gate"]), kind,
                     _np(v["w_post"]) if post else None, _np(v["w_pre"]) if pre else None,
                     _np(v["d_out"]) if with_out else None, _np(v["d_h"]) if pre else None, **KW)
    assert set(ref) == set(got)
    for name, (g, size) in ref.items():
        t = got[name]
        err = np.abs(_np(t) - g)
        assert (err <= _bf(t.dtype) * np.abs(g) + 2e-5 * size + 1e-30).all(), (name, err.max())
    first = {n: t.clone() for n, t in got.items()}
    call()
    for n, t in got.items():
        assert torch.equal(t, first[n]), n     # sums in a fixed order
    return got


@pytest.mark.parametrize("res,act", TYPES)
@pytest.mark.parametrize("H", [1, 7, 64, 250, 256, 1001, 2048, 4104])
def test_backward_sizes(H, res, act):
    _backward(37, H, res, act, "channel", True, True)


@pytest.mark.parametrize("res,act", TYPES)
@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("H", [96, 101])
def test_backward_kinds(H, post, pre, kind, res, act):
    _backward(50, H, res, act, kind, post, pre)


@pytest.mark.parametrize("T", [1, 2, 152, 153, 1300])
def test_backward_tokens(T):
    _backward(T, 256, BF16, BF16, "token", True, True)


@pytest.mark.parametrize("H,res,act", [(7168, BF16, BF16), (8192, F32, BF16), (9001, BF16, BF16),
                                       (10240, F32, F32)])
def test_backward_wide(H, res, act):
    _backward(4, H, res, act, "token", True, True)


def test_backward_strides_branches_and_missing_gradients():
    _backward(23, 64, BF16, BF16, "full", True, True, ld=67)
    _backward(23, 64, BF16, BF16, "full", True, True, ld=72)
    _backward(23, 64, BF16, BF16, "none", False, True, branch=False)
    _backward(23, 64, BF16, BF16, "token", True, True, with_out=False)


def test_another_stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _forward(64, 256, BF16, BF16, "none", True, True)
        _backward(64, 256, BF16, BF16, "channel", True, True)
