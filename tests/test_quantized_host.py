"""What `quantized` refuses: weights that are not what their addresses are read as.  No GPU."""
import dataclasses

import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K

H, E, I, S = 256, 8, 128, 192  # noqa: E741


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _weights(**kw):
    w = K.BlockWeights(bf(H), bf(H), bf(H), bf(H), bf(E, H), bf(E, 2 * I, H), bf(E, H, I), bf(2 * S, H), bf(H, S),
                       torch.zeros(E))
    return dataclasses.replace(w, **kw)


@pytest.mark.parametrize("name,t", [
    ("w_down", bf(E, I, H).transpose(1, 2)),              # a checkpoint's layout as a view
    ("w_gate_up", bf(E, H, 2 * I).transpose(1, 2)),
    ("w_gate_up", torch.zeros(E, 2 * I, H)),              # fp32
    ("w_down", torch.zeros(E, H, I, dtype=torch.float16)),
    ("w_down", bf(E, H, 2 * I)[..., :I]),                 # every other piece of a row
    ("w_gate_up", bf(1, 2 * I, H).expand(E, -1, -1)),     # fewer bytes than it seems
    ("w_gate_up", bf(E, I, H)), ("w_gate_up", bf(E - 1, 2 * I, H)), ("w_gate_up", bf(E, 2 * I, H - 8)),
    ("w_gate_up", bf(E * 2 * I, H)), ("w_gate_up", None), ("w_down", bf(1)[0]),
    ("w_down", bf(E, H, 0)),
    ("w_down", bf(E - 1, H, I)), ("w_down", bf(H, I)), ("w_down", None),
    ("w_down", torch.zeros(E, H, I, dtype=torch.bfloat16, device="meta")),
])
def test_experts_of_another_kind_are_refused(name, t):
    for shared in (False, True):
        with pytest.raises(ValueError, match=name):
            K.quantized(_weights(**{name: t}), "int4", 32, shared)


@pytest.mark.parametrize("name,t", [
    ("shared_down", bf(S, H).t()), ("shared_gate_up", bf(H, 2 * S).t()), ("shared_down", torch.zeros(H, S)),
    ("shared_gate_up", bf(2 * S + 2, H)), ("shared_down", bf(1, H, S)), ("shared_down", None),
    ("shared_gate_up", None)])
def test_a_shared_expert_of_another_kind_is_refused(name, t):
    with pytest.raises(ValueError, match=name):
        K.quantized(_weights(**{name: t}), shared=True)


def test_weights_in_host_memory_or_packed_already_are_refused():
    with pytest.raises(ValueError, match="on cuda wanted"):
        K.quantized(_weights(), shared=True)
    with pytest.raises(ValueError, match="on cuda wanted"):       # this one stays in bf16
        K.quantized(_weights(shared_down=None))
    with pytest.raises(ValueError, match="packed already"):
        K.quantized(_weights(quant=B.QuantWeights("e2m1", 16)))
    with pytest.raises(ValueError, match="router"):
        K.quantized(_weights(router=bf(E * H)))


@pytest.mark.parametrize("packed", [False, True])
def test_a_layer_that_names_its_shared_expert(monkeypatch, packed):
    """The shared expert in bf16 is the block's own step: the layer's calls get no I_shared."""
    layer = B.LayerDesc(T=20, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=3, I_shared=S)
    w = _weights()
    if packed:
        size = lambda *s: torch.zeros(B.moe_quant_size(B.QuantDesc(*s, "e2m1", 16)), dtype=torch.uint8)  # noqa: E731
        w = dataclasses.replace(w, w_gate_up=None, w_down=None,
                                quant=B.QuantWeights("e2m1", 16, size(2 * E, I, H), size(E, H, I)))
    block = K.MoeBlock(layer, B.GroupRoute(), w, device="cpu")
    assert block.shared == S and block.workspace.numel() >= B.moe_workspace_size(dataclasses.replace(layer, I_shared=0))
    descs = []
    for name in B.EXPORTS:
        monkeypatch.setattr(B, name, lambda d, *a: descs.append(d) or 0)
    block.forward(torch.zeros(5, H), bf(5, H), torch.ones(5, dtype=torch.int32))
    layers = [d for d in descs if isinstance(d, B.MoeLayerDesc)]
    assert len(layers) == 4 and all(d.I_shared == 0 and d.T == 5 for d in layers)
