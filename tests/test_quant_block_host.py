"""The decoder block with 4-bit experts, on the host: checks and buffers.  No GPU."""
import dataclasses

import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K

H, E, I, S = 256, 8, 128, 192  # noqa: E741


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


def _packed(*shape, group=16):
    return torch.zeros(B.moe_quant_size(B.QuantDesc(*shape, "int4", group)), dtype=torch.uint8)


def _weights(shared, **quant):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    q = dict(gate_up=_packed(2 * E, I, H), down=_packed(E, H, I))
    if shared:
        q.update(shared_gate_up=_packed(2, S, H), shared_down=_packed(1, H, S))
    q.update(quant)
    return K.BlockWeights(bf(H), bf(H), bf(H), bf(H), bf(E, H), None, None,
                          None if shared else bf(2 * S, H), None if shared else bf(H, S),
                          torch.zeros(E), B.QuantWeights("int4", 16, **q))


def _layer(T=20, **kw):
    return B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=3, **kw)


@pytest.mark.parametrize("shared", [False, True])
def test_workspace_does_for_a_step_of_any_size(shared):
    layer = _layer(300, I_shared=S if shared else 0)
    block = K.MoeBlock(layer, B.GroupRoute(), _weights(shared), device="cpu")
    assert block.shared == S and block.shared_packed == shared
    for t in range(301):
        assert B.moe_quant_workspace_size(dataclasses.replace(layer, T=t)) <= block.workspace.numel()


@pytest.mark.parametrize("bad", [
    dict(gate_up=torch.zeros(100, dtype=torch.uint8)), dict(down=None),
    dict(gate_up=_packed(2 * E, I, H).view(torch.int8)), dict(shared_down=_packed(1, H, S, group=32))])
def test_packed_weights_of_another_size_are_refused(bad):
    with pytest.raises(ValueError):
        K.MoeBlock(_layer(I_shared=S), B.GroupRoute(), _weights(True, **bad), device="cpu")


def test_a_packed_shared_expert_takes_no_adapters():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    pool = K.Adapters(bf(2, 8, H), bf(2, 2 * S, 8), bf(2, 8, S), bf(2, H, 8),
                      torch.full((2,), 8, dtype=torch.int32), torch.ones(2))
    with pytest.raises(ValueError):
        K.MoeBlock(_layer(I_shared=S), B.GroupRoute(), _weights(True), pool, device="cpu")
    block = K.MoeBlock(_layer(), B.GroupRoute(), _weights(False), pool, device="cpu")
    assert block.adapters is pool


@pytest.mark.parametrize("shared", [False, True])
def test_the_calls_of_a_step(monkeypatch, shared):
    calls = []
    for name in B.EXPORTS:
        monkeypatch.setattr(B, name, lambda *a, n=name: calls.append((n, a)) or 0)
    monkeypatch.setattr(B, "moe_lora_workspace_size", lambda d: 256)
    monkeypatch.setattr(B, "moe_quant_size", lambda d: B.lib().moe_quant_size(d.c()))
    block = K.MoeBlock(_layer(I_shared=S if shared else 0), B.GroupRoute(), _weights(shared), device="cpu")
    block.forward(torch.zeros(5, H), torch.zeros(5, H, dtype=torch.bfloat16), torch.ones(5, dtype=torch.int32))
    names = [n for n, _ in calls]
    if shared:
        assert names == ["moe_block_norm", "moe_layer_forward_quant", "moe_block_norm"]
        d = calls[1][1][0]
        assert (d.T, d.I_shared) == (5, S)
    else:
        assert names == ["moe_block_norm", "moe_route_groups", "moe_permute", "moe_grouped_ffn_quant",
                         "moe_lora_project", "moe_lora_project", "moe_combine", "moe_block_norm"]
