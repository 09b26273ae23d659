"""What the calls on 4-bit weights refuse on the host, without a GPU."""
import pytest

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


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), INVALID), (dict(rows=0), INVALID), (dict(K=0), INVALID), (dict(K=12), SHAPE),
    (dict(group=64), SHAPE), (dict(group=0), SHAPE), (dict(rows=(1 << 20) + 1), SHAPE),
])
def test_packing(kw, code):
    d = B.QuantDesc(**{**dict(count=2, rows=64, K=64), **kw})
    assert B.moe_quant_size(d) == 0
    assert B.moe_quant_pack(d, FAKE, FAKE, FAKE, FAKE, FAKE, 0) == code
    assert B.moe_quant_quantize(d, FAKE, FAKE, FAKE, 0) == code
    assert B.moe_quant_unpack(d, FAKE, FAKE, 0) == code


def test_packing_pointers_and_sizes():
    d = B.QuantDesc(2, 64, 64)
    for i in range(5):
        args = [FAKE] * 5
        args[i] = None
        assert B.moe_quant_pack(d, *args, 0) == INVALID
    assert B.moe_quant_pack(d, FAKE, FAKE, FAKE, FAKE + 8, FAKE, 0) == INVALID
    assert B.moe_quant_quantize(d, FAKE + 2, FAKE, FAKE, 0) == INVALID
    assert B.moe_quant_unpack(d, FAKE, None, 0) == INVALID
    c = d.c()
    c.code = 2
    assert B.moe_quant_size(c) == 0 and B.moe_quant_pack(c, *[FAKE] * 5, 0) == INVALID
    # a tile is 8192 bytes of codes and 8 or 4 scales for each of 128 rows, a factor behind all
    assert B.moe_quant_size(B.QuantDesc(1, 1, 8, "e2m1", 16)) == 9216 + 256
    assert B.moe_quant_size(B.QuantDesc(64, 129, 136, "int4", 32)) == 64 * 4 * 8704 + 256


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(K=12), SHAPE),
    (dict(ldx=32), INVALID), (dict(ldx=68), SHAPE), (dict(ldy=100), INVALID), (dict(group=8), SHAPE),
    (dict(N=129, swiglu=True), SHAPE), (dict(T=(1 << 23) + 1), SHAPE),
])
def test_project(kw, code):
    d = B.QuantProject(**{**dict(T=4, K=64, N=128), **kw})
    assert B.moe_quant_project_workspace_size(d) == 0
    assert B.moe_quant_project(d, FAKE, FAKE, FAKE, FAKE, WS, 0) == code


def test_project_pointers():
    d = B.QuantProject(4, 64, 128)
    for i, bad in ((0, None), (0, FAKE + 8), (1, None), (1, FAKE + 4), (2, None), (2, FAKE + 1), (3, None),
                   (3, FAKE + 2)):
        args = [FAKE] * 4
        args[i] = bad
        assert B.moe_quant_project(d, *args, WS, 0) == INVALID
    assert B.moe_quant_project(d, *[FAKE] * 4, None, 0) == WORKSPACE
    assert B.moe_quant_project(d, *[FAKE] * 4, WS + 16, 0) == WORKSPACE
    assert B.moe_quant_project(B.QuantProject(0, 64, 128), *[None] * 4, None, 0) == 0


def _desc(**kw):
    return B.LayerDesc(**{**dict(T=64, H=256, n_experts=16, n_sub=4, I_sub=128, k_max=8), **kw})


def _weights(**kw):
    return B.QuantWeights(**{**dict(code="e2m1", group=16, gate_up=FAKE, down=FAKE), **kw})


def _layer(d=None, w=None, groups=None, x=FAKE, router=FAKE, k=FAKE, load=None, out=FAKE, st=FAKE, ws=WS):
    return B.moe_layer_forward_quant(d or _desc(), groups, w or _weights(), x, router, k, load, out, st, ws, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(d=_desc(H=100)), SHAPE), (dict(d=_desc(T=-1)), INVALID), (dict(d=_desc(k_max=33)), SHAPE),
    (dict(d=_desc(I_shared=-64)), INVALID), (dict(d=_desc(I_shared=100)), SHAPE),
    (dict(d=_desc(I_sub=(1 << 20) + 64)), SHAPE),
    (dict(d=_desc(I_shared=64)), INVALID),               # no packed shared expert
    (dict(d=_desc(I_shared=64), w=_weights(shared_gate_up=FAKE)), INVALID),
    (dict(w=_weights(gate_up=None)), INVALID), (dict(w=_weights(down=FAKE + 8)), INVALID),
    (dict(w=_weights(group=64)), SHAPE),
    (dict(groups=B.GroupRoute(n_groups=7)), SHAPE), (dict(groups=B.GroupRoute(group_best=3)), INVALID),
    (dict(load=FAKE), INVALID),                          # loads are the group router's
    (dict(groups=B.GroupRoute(), load=FAKE + 2), INVALID),
    (dict(x=None), INVALID), (dict(router=FAKE + 8), INVALID), (dict(k=None), INVALID),
    (dict(out=None), INVALID), (dict(st=None), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=WS + 128), WORKSPACE), (dict(d=_desc(T=0)), 0),
])
def test_layer(kw, code):
    assert _layer(**kw) == code


def test_ffn_calls():
    w = _weights()
    args = [FAKE] * 5
    for i in range(5):
        bad = list(args)
        bad[i] = None
        assert B.moe_grouped_ffn_quant(_desc(), w, *bad, WS, 0) == INVALID
    assert B.moe_grouped_ffn_quant(_desc(), w, *args, None, 0) == WORKSPACE
    assert B.moe_grouped_ffn_quant(_desc(T=0), w, *[None] * 5, None, 0) == 0
    assert B.moe_grouped_ffn_quant(_desc(I_sub=96), w, *args, WS, 0) == SHAPE
    d = _desc(I_shared=64)
    assert B.moe_shared_ffn_quant(_desc(), w, FAKE, FAKE, FAKE, WS, 0) == INVALID
    assert B.moe_shared_ffn_quant(d, w, FAKE, FAKE, FAKE, WS, 0) == INVALID
    s = _weights(gate_up=None, down=None, shared_gate_up=FAKE, shared_down=FAKE)
    assert B.moe_shared_ffn_quant(d, s, None, FAKE, FAKE, WS, 0) == INVALID
    assert B.moe_shared_ffn_quant(d, s, FAKE, FAKE, FAKE, WS + 1, 0) == WORKSPACE
    assert B.moe_quant_workspace_size(_desc(H=32)) == 0
    assert B.moe_quant_workspace_size(d) >= B.moe_quant_workspace_size(_desc()) > B.moe_workspace_size(_desc())
