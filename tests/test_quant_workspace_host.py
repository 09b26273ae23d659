"""What the calls on 4-bit weights take beside the bf16 layer's workspace.  No GPU."""
import os

import pytest

from aware_moe_expert_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


@pytest.mark.parametrize("T,H,E,I,k,shared", [(1, 64, 1, 64, 1, 0), (4, 2048, 256, 384, 16, 128), (9, 64, 8, 4096, 8, 0),
                                              (300, 320, 12, 192, 3, 64), (8192, 2048, 128, 768, 8, 0),
                                              (16384, 7168, 256, 2048, 8, 2048)])
def test_the_experts_fp32_rows_take_none(T, H, E, I, k, shared):  # noqa: E741
    """16384 tokens of 8 units and H 7168 are 3.8 GB of them, in the place of the bf16 layer's rows."""
    shape = dict(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=k)
    bf16 = B.moe_workspace_size(B.LayerDesc(**shape, I_shared=shared, w_shared_gate_up=1 << 20, w_shared_down=1 << 20))
    quant = B.moe_quant_workspace_size(B.LayerDesc(**shape, I_shared=shared))
    few = 2 if T <= 4 else 1                    # the activations, as two bf16 up to four tokens
    want = few * T * k * I * 2 + (T * H * 4 + (few - 1) * T * shared * 2 if shared else 0)
    assert bf16 > 0 and want <= quant - bf16 <= want + 4 * 256
