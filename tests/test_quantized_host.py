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
