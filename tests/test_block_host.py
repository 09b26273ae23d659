"""What the decoder block does on the host: its buffers, its checks, the streams
and arguments it hands to the library.  No GPU: the buffers are host memory, and
where a step runs, the library's calls are recorded instead of made."""
import dataclasses

import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


def _block(T=64, H=256, experts=32, I=128, k=6, shared=64, n_adapters=6, rank=16,  # noqa: E741
           groups=None):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    w = K.BlockWeights(bf(H), bf(H), bf(H), bf(H), bf(experts, H), bf(experts, 2 * I, H),
                       bf(experts, H, I), bf(2 * shared, H), bf(H, shared), torch.zeros(experts))
    pool = K.Adapters(bf(n_adapters, rank, H), bf(n_adapters, 2 * shared, rank),
                      bf(n_adapters, rank, shared), bf(n_adapters, H, rank),
                      torch.full((n_adapters,), rank, dtype=torch.int32), torch.ones(n_adapters))
    layer = B.LayerDesc(T=T, H=H, n_experts=experts, n_sub=1, I_sub=I, k_max=k)
    return K.MoeBlock(layer, groups or B.GroupRoute(), w, pool, device="cpu")


@pytest.mark.parametrize("T,H,experts,I,k", [
    (342, 256, 32, 128, 6),      # a step of 341 tokens needs 8 MB more than one of 342
    (147, 2048, 64, 512, 8),
    (600, 128, 64, 64, 8), (1, 64, 8, 64, 2)])
def test_the_workspace_does_for_a_step_of_any_size(T, H, experts, I, k):  # noqa: E741
    block = _block(T, H, experts, I, k)
    for t in range(1, T + 1):
        d = dataclasses.replace(block.layer, T=t)
        assert B.moe_workspace_size(d) <= block.workspace.numel(), t
        for first in (True, False):
            assert B.moe_lora_workspace_size(block._lora(t, first)) <= block.lora_workspace.numel()
