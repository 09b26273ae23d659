"""The block norms over more rows than a launch has row groups, against the float64
forms and with the tolerances of the tests of single rows."""
import pytest
import test_gpu_block_norm as rows
import torch
from test_block_norm_plan import plan
from test_gpu_block_norm import _backward, _forward

from aware_moe_expert_gb300 import binding as B

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


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _rows(T, H, res, act, kind, back, aligned=True):
    """Rows of the launch's busiest row group, and its slots."""
    grid, groups, slots, _ = plan(B.lib(), B.BlockNormDesc(T=T, H=H, residual_dtype=res, act_dtype=act,
                                                           gate=kind), back, aligned, _sms())
    return -(-T // (grid * groups)), slots


def _off_the_grid(monkeypatch, names=("y",)):
    """Inputs one element off the 16-byte grid: columns are taken one at a time."""
    make = rows._make

    def moved(*args, **kw):
        v = make(*args, **kw)
        for n in names:
            t = v[n]
            buf = torch.zeros(t.untyped_storage().nbytes() // t.element_size() + 9, dtype=t.dtype, device="cuda")
            v[n] = torch.as_strided(buf, t.shape, t.stride(), 1)
            v[n].copy_(t)
        return v
    monkeypatch.setattr(rows, "_make", moved)


# widths of every variant: one warp a row, eight columns a thread, 24 columns; whole
# pieces, pieces that begin before the row, one column at a time; one slot and several
FORWARD = [
    (20000, 64, BF16, BF16, "full"), (20000, 101, BF16, BF16, "channel"), (17000, 256, F32, BF16, "none"),
    (16000, 250, F32, F32, "token"), (14000, 512, BF16, BF16, "full"), (5000, 1001, F32, BF16, "channel"),
    (4000, 2048, F32, F32, "full"), (3000, 2001, BF16, BF16, "none"), (1000, 7168, BF16, BF16, "token"),
    (1000, 7929, BF16, BF16, "full"), (900, 8192, BF16, BF16, "full"), (700, 8193, F32, BF16, "channel"),
    (700, 12288, F32, F32, "none"), (600, 16384, F32, F32, "channel"), (600, 16383, F32, F32, "none"),
    (700, 16383, BF16, BF16, "token")]


@pytest.mark.parametrize("T,H,res,act,kind", FORWARD)
def test_forward_many_rows_a_group(T, H, res, act, kind):
    n, slots = _rows(T, H, res, act, kind, 0)
    assert n >= 3 and n > slots      # a slot is filled again
    _forward(T, H, res, act, kind, True, True)


@pytest.mark.parametrize("T,H,res,act,kind", FORWARD[::3] + [(700, 12288, BF16, BF16, "full")])
def test_forward_many_rows_a_group_off_the_grid(monkeypatch, T, H, res, act, kind):
    assert _rows(T, H, res, act, kind, 0, False)[0] >= 3
    _off_the_grid(monkeypatch)
    _forward(T, H, res, act, kind, True, True)


@pytest.mark.parametrize("H,ld", [(64, 72), (101, 107), (2001, 2011), (1024, 1029)])
@pytest.mark.parametrize("post,pre,branch", [(True, True, True), (False, True, True),
                                             (True, False, True), (False, True, False)])
def test_forward_many_strided_rows(H, ld, post, pre, branch):
    T = 20000 if H < 1000 else 5000
    _forward(T, H, BF16, BF16, "none", post, pre, ld=ld, branch=branch)


BACKWARD = [
    (14000, 64, BF16, BF16, "full"), (14000, 101, BF16, BF16, "channel"), (14000, 256, F32, BF16, "none"),
    (9000, 250, F32, F32, "token"), (6000, 512, BF16, BF16, "full"), (4000, 1001, F32, BF16, "channel"),
    (2500, 2048, BF16, BF16, "token"), (2500, 2048, F32, F32, "full"), (2000, 2001, BF16, BF16, "none"),
    (1000, 4096, BF16, BF16, "channel"), (1000, 7168, BF16, BF16, "token"), (700, 8192, F32, BF16, "full"),
    (700, 9001, BF16, BF16, "channel"), (600, 10240, F32, F32, "token"), (500, 16384, BF16, BF16, "none")]


@pytest.mark.parametrize("T,H,res,act,kind", BACKWARD)
def test_backward_many_rows_a_group(T, H, res, act, kind):
    n, slots = _rows(T, H, res, act, kind, 1)
    assert n >= 3 and n > slots
    _backward(T, H, res, act, kind, True, True)


@pytest.mark.parametrize("T,H,res,act,kind", BACKWARD[::3])
def test_backward_many_rows_a_group_off_the_grid(monkeypatch, T, H, res, act, kind):
    _off_the_grid(monkeypatch, ("y", "d_h"))
    _backward(T, H, res, act, kind, True, True)


@pytest.mark.parametrize("post,pre,branch,with_out", [
    (True, False, True, True), (False, True, True, True), (False, True, False, True),
    (True, True, True, False)])
def test_backward_many_rows_parts_left_out(post, pre, branch, with_out):
    _backward(3000, 1024, BF16, BF16, "token" if branch else "none", post, pre, ld=1032, branch=branch,
              with_out=with_out)
