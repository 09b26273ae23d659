"""The decoder block on a stream given as an argument."""
import pytest
import torch

from aware_moe_expert_gb300 import block as K

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_steps_and_balancing_on_a_given_stream(handle):
    """Steps on a side stream while the current stream allocates and writes memory:
    the same results and biases as on one stream."""
    def run(stream, disturb):
        block, residual, attn, k, adapter = K.synthetic(T=256, seed=11)
        torch.cuda.synchronize()
        work = [residual.clone() for _ in range(8)]
        torch.cuda.synchronize()
        outs = []
        for r in work:
            outs.append(block.forward(r, attn, k, adapter, stream=stream).clone()
                        if stream is None else block.forward(r, attn, k, adapter, stream=stream))
            block.balance(0.01, stream=stream)
            if disturb:
                for _ in range(4):
                    torch.full_like(attn, float("nan"))
        torch.cuda.synchronize()
        assert block.device_status(stream) == 0
        return outs, block.weights.select_bias

    s = torch.cuda.Stream()
    want, bias = run(None, False)
    got, bias2 = run(s.cuda_stream if handle else s, True)
    assert torch.equal(bias, bias2) and all(torch.equal(a, b) for a, b in zip(want, got))
    assert (bias != 0).any()


def test_the_result_belongs_to_the_given_stream():
    """Memory of a result that was dropped is used again on its own stream only."""
    block, residual, attn, k, adapter = K.synthetic(T=64, seed=12)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    at = block.forward(residual, attn, k, adapter, stream=s).data_ptr()   # dropped at once
    mine = [torch.empty_like(attn) for _ in range(8)]
    assert at not in [t.data_ptr() for t in mine]
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        again = torch.empty_like(attn)
    assert again.data_ptr() == at


def test_a_step_of_fewer_tokens_that_needs_more_workspace():
    """342 tokens need 19.8 MB, 341 need 28.1 MB."""
    block, residual, attn, k, adapter = K.synthetic(T=342, seed=13)
    a = block.forward(residual[:341].clone(), attn[:341], k[:341], adapter[:341])
    b = K.synthetic(T=341, seed=13)[0].forward(residual[:341].clone(), attn[:341], k[:341],
                                               adapter[:341])
    assert block.device_status() == 0 and torch.equal(a, b)


def test_a_step_without_adapter_indexes():
    block, residual, attn, k, _ = K.synthetic(T=40, seed=14)
    a = block.forward(residual.clone(), attn, k)
    block.adapters = None
    b = block.forward(residual.clone(), attn, k)
    assert block.device_status() == 0 and torch.equal(a, b)


def test_rows_at_a_stride_and_no_tokens():
    block, residual, attn, k, adapter = K.synthetic(T=40, seed=15)
    want_r = residual.clone()
    want = block.forward(want_r, attn, k, adapter)
    wide = torch.full((40, 300), 7.0, device="cuda")
    wide[:, :256] = residual
    apart = torch.zeros(40, 264, device="cuda", dtype=torch.bfloat16)
    apart[:, :256] = attn
    got = block.forward(wide[:, :256], apart[:, :256], k, adapter)
    # another order of a row's sums: the layer's tolerance
    assert (got.float() - want.float()).abs().max() <= 1e-2 + 1e-2 * want.float().abs().max()
    assert torch.allclose(wide[:, :256], want_r, rtol=1e-2, atol=1e-2) and (wide[:, 256:] == 7).all()
    assert block.forward(residual[:0], attn[:0], k[:0], adapter[:0]).shape == (0, 256)
    assert (block.load == 0).all() and block.device_status() == 0
