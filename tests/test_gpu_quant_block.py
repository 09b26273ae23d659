"""The decoder block with 4-bit experts: a run of routing, experts, shared expert and
norms as they are used, against the same block on the unpacked weights."""
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K

pytestmark = pytest.mark.gpu

# A rounding to bf16 moves a value by up to 2^-8 of it: 2^-8 / sqrt(3) in the mean square
# at the most.  The two blocks differ by nine that are independent of one another: the
# unpacked gate, up and down weights (the code times the scale is exact in bf16, times
# the factor it is not), and in each block the activations, the rows and their sum.  A
# sum over many products carries a relative change of its terms on in the mean square;
# silu's slope (1.1 at the most) and the product with `up` are within that bound, as a
# rounding's mean square is 0.72 of it over a value's whole range.
ROUND = 2.0 ** -8 / 3 ** 0.5
CHANGE = 9 ** 0.5 * ROUND


def _unpack(packed, count, rows, K_, q):
    w = torch.empty(count, rows, K_, dtype=torch.bfloat16, device="cuda")
    B.check(B.moe_quant_unpack(B.QuantDesc(count, rows, K_, q.code, q.group), packed, w))
    return w


def _bf16_block(block):
    """A block of the same layer on the unpacked weights."""
    w, layer, q = block.weights, block.layer, block.weights.quant
    E, H, I, S = layer.E_r, layer.H, layer.I_sub, block.shared  # noqa: E741
    gu, dn = w.shared_gate_up, w.shared_down
    if block.shared_packed:
        gu, dn = _unpack(q.shared_gate_up, 2, S, H, q).view(2 * S, H), _unpack(q.shared_down, 1, H, S, q)[0]
    plain = K.BlockWeights(w.attn_post_norm, w.pre_norm, w.ffn_post_norm, w.next_pre_norm, w.router,
                           _unpack(q.gate_up, 2 * E, I, H, q).view(E, 2 * I, H), _unpack(q.down, E, H, I, q),
                           gu, dn, w.select_bias.clone())
    layer = B.LayerDesc(T=layer.T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=layer.k_max,
                        score=layer.score, renorm=layer.renorm, route_scale=layer.route_scale)
    return K.MoeBlock(layer, block.groups, plain, block.adapters)


@pytest.mark.parametrize("T", [1, 7, 64, 300])
@pytest.mark.parametrize("quant,group,shared", [("e2m1", 16, False), ("int4", 32, True), ("e2m1", 32, True)])
def test_steps_like_those_of_the_unpacked_block(T, quant, group, shared):
    block, residual, attn, k, adapter = K.synthetic(T=T, seed=T, quant=quant, group=group, shared_quant=shared)
    other = _bf16_block(block)
    adapter = None if shared else adapter
    r1, r2 = residual.clone(), residual.clone()
    scale = block.weights.ffn_post_norm.abs().float()
    for _ in range(3):
        a, b = block.forward(r1, attn, k, adapter), other.forward(r2, attn, k, adapter)
        assert torch.equal(block.load, other.load)
        d = (r1 - r2) / scale
        # the post norm's output is of size one times its weight, and six deviations
        # of CHANGE are passed once in 5e8 elements
        assert float(d.square().mean().sqrt()) <= CHANGE and float(d.abs().max()) <= 6 * CHANGE
        # the normed output rounds once more in each block
        assert float((a.float() - b.float()).norm()) <= (CHANGE ** 2 + 2 * ROUND ** 2) ** 0.5 * float(b.float().norm())
        r2.copy_(r1)
        block.balance()
        other.balance()
    assert block.device_status() == 0 and other.device_status() == 0


@pytest.mark.parametrize("shared", [False, True])
def test_in_a_graph_and_on_a_stream(shared):
    block, residual, attn, k, adapter = K.synthetic(T=48, seed=5, quant="e2m1", shared_quant=shared)
    adapter = None if shared else adapter
    want = [block.forward(residual[:t].clone(), attn[:t], k[:t], None if shared else adapter[:t]).clone()
            for t in (48, 5)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t, w in zip((48, 5), want):
        got = block.forward(residual[:t].clone(), attn[:t], k[:t], None if shared else adapter[:t])
        assert torch.equal(got, w)
    work, g = residual.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block.forward(work, attn, k, adapter)
    work.copy_(residual)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    r = residual.clone()
    torch.cuda.synchronize()
    got = block.forward(r, attn, k, adapter, stream=s)
    s.synchronize()
    assert torch.equal(got, want[0]) and block.device_status(s) == 0


def test_quantized_refuses_weights_that_are_not_finite():
    block, *_ = K.synthetic(T=4)
    w = block.weights
    w.w_down[1, 2, 3] = float("nan")
    with pytest.raises(B.MoeError):
        K.quantized(w)
