"""What the group router, the block norms and the adapter projection refuse on
the host, without a GPU: nothing is enqueued before the arguments are checked."""
import pytest
import torch

from aware_moe_expert_gb300 import binding as B

FAKE, WS = 1 << 20, 1 << 21          # aligned, never dereferenced
INVALID, SHAPE, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


def _desc(**kw):
    base = dict(T=64, H=256, n_experts=16, n_sub=4, I_sub=128, k_max=8)
    base.update(kw)
    return B.LayerDesc(**base)


def _route(desc=None, x=FAKE, w=FAKE, logits=None, k=FAKE, idx=FAKE, tw=FAKE, load=None, st=FAKE,
           ws=WS, **g):
    groups = dict(n_groups=8, groups_kept=4, group_best=2)
    groups.update(g)
    return B.moe_route_groups(desc or _desc(), B.GroupRoute(**groups), x, w, logits, k, None, idx,
                              tw, None, load, st, ws, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(n_groups=0), INVALID), (dict(groups_kept=0), INVALID), (dict(groups_kept=9), INVALID),
    (dict(group_best=3), INVALID), (dict(group_best=0), INVALID),
    (dict(n_groups=7), SHAPE),                       # does not divide 64 units
    (dict(n_groups=64, groups_kept=7), SHAPE),       # 7 units kept, k_max 8
    (dict(select_bias=FAKE + 2), INVALID),
    (dict(desc=_desc(H=100)), SHAPE), (dict(desc=_desc(T=-1)), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(k=None), INVALID),
    (dict(idx=None), INVALID), (dict(tw=FAKE + 1), INVALID), (dict(load=FAKE + 1), INVALID),
    (dict(st=None), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=WS + 16), WORKSPACE),
    (dict(logits=FAKE + 2), INVALID),
    (dict(desc=_desc(T=0)), 0),
])
def test_group_router(kw, code):
    assert _route(**kw) == code


def test_route_backward_and_layer():
    d = _desc()
    assert B.moe_route_backward(d, None, FAKE, FAKE, FAKE, FAKE, 0) == INVALID
    assert B.moe_route_backward(d, FAKE, FAKE, FAKE, FAKE + 2, FAKE, 0) == INVALID
    assert B.moe_route_backward(_desc(k_max=40), FAKE, FAKE, FAKE, FAKE, FAKE, 0) == SHAPE
    assert B.moe_route_backward(_desc(T=0), None, None, None, None, None, 0) == 0
    g = B.GroupRoute(n_groups=8, groups_kept=4)
    args = [FAKE] * 5
    assert B.moe_layer_forward_groups(d, g, *args, None, FAKE, FAKE, None, 0) == WORKSPACE
    assert B.moe_layer_forward_groups(d, g, None, *args[1:], None, FAKE, FAKE, WS, 0) == INVALID
    assert B.moe_layer_forward_groups(d, B.GroupRoute(n_groups=5), *args, None, FAKE, FAKE, WS,
                                      0) == SHAPE
    assert B.moe_layer_forward_groups(_desc(T=0), g, *args, None, FAKE, FAKE, WS, 0) == 0


def _norm(r=FAKE, y=FAKE, gate=None, kind="none", out=FAKE, h=FAKE, **kw):
    base = dict(T=4, H=64, w_post=FAKE, w_pre=FAKE, gate=kind)
    base.update(kw)
    return B.moe_block_norm(B.BlockNormDesc(**base), r, y, gate, out, h, 0)


F32 = torch.float32


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=16385), SHAPE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(ld_branch=63), INVALID), (dict(ld_out=-64), INVALID),
    (dict(act_dtype=F32), SHAPE),                                 # fp32 branch, bf16 residual
    (dict(r=None), INVALID), (dict(y=None), INVALID), (dict(out=None), INVALID),
    (dict(h=None), INVALID), (dict(w_pre=None), INVALID),         # h without its weight
    (dict(gate=FAKE), INVALID),                                   # a gate, and none in the desc
    (dict(r=FAKE + 1), INVALID), (dict(r=FAKE + 2, residual_dtype=F32), INVALID),
    (dict(T=0, r=None, y=None, out=None, h=None), 0),
])
def test_block_norm(kw, code):
    assert _norm(**kw) == code


def test_block_norm_gate_and_workspace():
    assert B.moe_block_norm(B.BlockNormDesc(T=4, H=64, gate="token"), FAKE, FAKE, None, FAKE, None,
                            0) == INVALID
    assert B.moe_block_norm(B.BlockNormDesc(T=4, H=64, gate="channel"), FAKE, None, FAKE, FAKE,
                            None, 0) == INVALID
    assert B.moe_block_norm_workspace_size(B.BlockNormDesc(T=4, H=0)) == 0
    n = B.moe_block_norm_workspace_size(B.BlockNormDesc(T=4, H=64))
    assert n >= 4 * 3 * 64 * 4 and n % 256 == 0


def _back(d=None, ws=WS, **kw):
    a = dict(r=FAKE, y=FAKE, gate=FAKE, do=None, dh=FAKE, dr=FAKE, dy=FAKE, dg=FAKE, dwp=FAKE,
             dwq=FAKE)
    a.update(kw)
    d = d or B.BlockNormDesc(T=4, H=64, gate="channel", w_post=FAKE, w_pre=FAKE)
    return B.moe_block_norm_backward(d, *a.values(), ws, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(r=None), INVALID), (dict(dr=None), INVALID), (dict(dy=None), INVALID),
    (dict(dg=None), INVALID), (dict(dwp=None), INVALID), (dict(dwq=None), INVALID),
    (dict(dh=None), INVALID), (dict(dg=FAKE + 2), INVALID), (dict(do=FAKE + 1), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=WS + 8), WORKSPACE),
    (dict(d=B.BlockNormDesc(T=4, H=16384, residual_dtype=F32, act_dtype=F32, gate="channel",
                            w_post=FAKE, w_pre=FAKE)), SHAPE),
])
def test_block_norm_backward(kw, code):
    assert _back(**kw) == code


def _lora(x=FAKE, w=FAKE, a=FAKE, b=FAKE, ranks=FAKE, scales=FAKE, idx=FAKE, y=FAKE, st=FAKE,
          ws=WS, **kw):
    base = dict(T=4, K=64, N=48, n_adapters=2, r_max=8)
    base.update(kw)
    return B.moe_lora_project(B.LoraDesc(**base), x, w, a, b, ranks, scales, idx, y, st, ws, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(r_max=0), INVALID),
    (dict(n_adapters=-1), INVALID), (dict(ldx=32), INVALID), (dict(ldy=47), INVALID),
    (dict(K=60), SHAPE), (dict(ldx=68), SHAPE), (dict(r_max=12), SHAPE), (dict(r_max=136), SHAPE),
    (dict(N=47, swiglu=True), SHAPE),
    (dict(x=None), INVALID), (dict(x=FAKE + 2), INVALID), (dict(w=None), INVALID),
    (dict(a=None), INVALID), (dict(b=FAKE + 8), INVALID), (dict(ranks=None), INVALID),
    (dict(scales=None), INVALID), (dict(idx=FAKE + 2), INVALID), (dict(y=None), INVALID),
    (dict(y=FAKE + 1), INVALID), (dict(st=None), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=WS + 64), WORKSPACE), (dict(T=0), 0),
])
def test_lora_project(kw, code):
    assert _lora(**kw) == code


def test_lora_workspace_size():
    assert B.moe_lora_workspace_size(B.LoraDesc(T=4, K=60, N=48, n_adapters=2, r_max=8)) == 0
    n = B.moe_lora_workspace_size(B.LoraDesc(T=4, K=64, N=48, n_adapters=2, r_max=8))
    assert n > 0 and n % 256 == 0
