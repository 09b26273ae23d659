"""How the block norms are launched, worked out on the host: every width that the
library takes fits the shared memory of a CTA with its sum buffers and barriers."""
import ctypes

import pytest
import torch

from aware_moe_expert_gb300 import binding as B

BF16, F32 = torch.bfloat16, torch.float32
SHAPE, MOST = 2, 227 * 1024


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


def plan(lib, desc, back, aligned=True, sm=152):
    """(CTAs, groups, slots, shared memory) or None where the width is refused."""
    out = (ctypes.c_int32 * 4)()
    lib.moe_block_norm_plan.argtypes = [ctypes.POINTER(B.MoeNormDesc), ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.POINTER(ctypes.c_int32)]
    code = lib.moe_block_norm_plan(desc if isinstance(desc, B.MoeNormDesc) else desc.c(), back,
                                   aligned, sm, out)
    assert code in (0, SHAPE)
    return None if code else tuple(out)


@pytest.mark.parametrize("res,act", [(BF16, BF16), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("gate", ["none", "full"])
@pytest.mark.parametrize("back", [0, 1])
@pytest.mark.parametrize("sm", [148, 152])
def test_every_width_fits_a_cta(lib, res, act, gate, back, sm):
    d = B.BlockNormDesc(T=1, H=8, residual_dtype=res, act_dtype=act, gate=gate).c()
    widths = list(range(1, 1100)) + list(range(1100, 16385, 61)) + [4096, 7936, 8192, 16384]
    refused = []
    for d.H in widths:
        # as many row groups as there are rows for, from one to all that fit
        for d.T in [1] + [sm * g for g in range(1, 17)] + [100000]:
            for aligned in (1, 0):
                p = plan(lib, d, back, aligned, sm)
                if p is None:
                    refused.append(d.H)
                    continue
                grid, groups, slots, smem = p
                assert 0 < smem <= MOST, (d.H, d.T, p)
                assert 1 <= slots <= 4 and 1 <= groups <= 16 and 1 <= grid <= sm
                assert groups <= -(-d.T // sm) and grid * groups >= min(d.T, sm // 8 * 8)
    # refused: a row of every tensor read, as the 16-byte granules around it, over 200 KB
    full, size = gate == "full", {BF16: 2, F32: 4}
    rows, a_row = 2 + 2 * back + full, (1 + back) * size[res] + (1 + back + full) * size[act]
    assert all(a_row * (h + 7) + 47 * rows + 128 > 200 * 1024 for h in refused)


def test_a_misaligned_status_word_is_refused(lib):
    at = 1 << 20         # aligned, not dereferenced
    d = B.BlockNormDesc(T=4, H=64, w_pre=at, dev_status=at + 2)
    assert B.moe_block_norm(d, at, at, None, at, at, 0) == 1
    assert B.moe_block_norm_backward(d, at, at, None, at, at, at, at, None, None, at, at, 0) == 1
