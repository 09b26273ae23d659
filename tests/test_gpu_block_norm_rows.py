"""The block norms over more rows than a launch has row groups, against the float64
forms and with the tolerances of the tests of single rows."""
import pytest
import torch
from test_gpu_block_norm import _backward, _forward

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# widths whose row slots and sum buffers together fill the shared memory of a CTA
@pytest.mark.parametrize("T,H,res,act,kind", [
    (2500, 248, F32, F32, "full"), (2500, 346, F32, F32, "full"), (2500, 352, F32, F32, "full"),
    (2100, 384, F32, F32, "full"), (2128, 389, F32, F32, "full")])
def test_forward_where_shared_memory_is_full(T, H, res, act, kind):
    _forward(T, H, res, act, kind, True, True)


@pytest.mark.parametrize("T,H,res,act,kind", [
    (2500, 144, F32, F32, "full"), (2500, 192, F32, F32, "full"), (2281, 193, F32, F32, "full"),
    (2500, 184, F32, F32, "token"), (2500, 248, F32, F32, "channel"), (2500, 208, F32, BF16, "full"),
    (2500, 240, F32, BF16, "token"), (2500, 249, F32, BF16, "none"), (2100, 224, F32, F32, "full"),
    (2200, 208, F32, F32, "full")])
def test_backward_where_shared_memory_is_full(T, H, res, act, kind):
    _backward(T, H, res, act, kind, True, True)
