"""The decoder block made of the norms, the group router, the routed experts and
the adapted shared expert, against the float64 forms of its steps.

Each step is compared on the inputs that the step had on the GPU, so that one
step's rounding is not another's error: the layer tolerance of the routed and
shared outputs (1e-2 + 1e-2 |ref| per element, 5e-3 in the Frobenius norm), one
bf16 rounding of the norms' outputs.
"""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K
from oracle import block_norm as N
from oracle import group_route as G
from oracle import lora as L

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _close(got, ref):
    got = _np(got)
    assert (np.abs(got - ref) <= 1e-2 + 1e-2 * np.abs(ref)).all()
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref) + 1e-6


@pytest.mark.parametrize("T", [1, 7, 64, 300])
def test_block_steps(T):
    block, residual, attn, k, adapter = K.synthetic(T=T, seed=T)
    before = residual.clone()
    out = block.forward(residual, attn, k, adapter)
    assert block.device_status() == 0
    w = block.weights
    # attention post-norm, residual, pre-norm
    r1, h1, mag = N.forward(_np(before), _np(attn), None, "none", _np(w.attn_post_norm),
                            _np(w.pre_norm))
    h = block.h[:T]
    assert (np.abs(_np(h) - h1) <= 2.0 ** -8 * np.abs(h1) + 2e-5 * (np.abs(h1) + 1)).all()
    # routing on the block's own logits
    logits = block.logits[:T].cpu().numpy()
    bias = w.select_bias.cpu().numpy()
    hh, want = _np(h), np.zeros((T, h.shape[1]))
    gu, dn = _np(w.w_gate_up), _np(w.w_down)
    I = dn.shape[2]  # noqa: E741
    chosen_gpu = block.topk_idx[:T].cpu().numpy()
    load = np.zeros(len(bias), dtype=np.int64)
    for t in range(T):
        units, wt, gap = G.route_token(logits[t], int(k[t]), "sigmoid", True, 2.5, 8, 4, 2, bias)
        if gap > 2e-6:
            assert list(chosen_gpu[t][:len(units)]) == units
        else:
            units = [u for u in chosen_gpu[t] if u >= 0]
            s = 1 / (1 + np.exp(-logits[t][units].astype(np.float64)))
            wt = 2.5 * s / s.sum()
        load[units] += 1
        for u, g in zip(units, wt):
            a = gu[u, :I] @ hh[t]
            want[t] += g * (dn[u] @ (a / (1 + np.exp(-a)) * (gu[u, I:] @ hh[t])))
    assert (block.load.cpu().numpy() == load).all()
    # shared expert with adapters
    p, ad = block.adapters, adapter.cpu().numpy()
    pool = lambda a, b: (_np(a), _np(b), p.ranks.cpu().numpy(), _np(p.scales), ad)  # noqa: E731
    act, _, _ = L.project(hh, _np(w.shared_gate_up), *pool(p.gate_up_a, p.gate_up_b), swiglu=True)
    _close(block.act[:T], act)
    ys, _, _ = L.project(_np(block.act[:T]), _np(w.shared_down), *pool(p.down_a, p.down_b))
    _close(block.y_shared[:T], ys)
    _close(block.y[:T], want + _np(block.y_shared[:T]))
    # output norm, residual, next pre-norm
    r2, h2, mag2 = N.forward(r1, _np(block.y[:T]), None, "none", _np(w.ffn_post_norm),
                             _np(w.next_pre_norm))
    assert (np.abs(_np(residual) - r2) <= 2e-5 * (mag + mag2)).all()
    assert (np.abs(_np(out) - h2) <= 2.0 ** -8 * np.abs(h2) + 4e-5 * (np.abs(h2) + 1)).all()


def test_smaller_steps_without_adapters_and_on_a_stream():
    block, residual, attn, k, _ = K.synthetic(T=64)
    block.adapters = None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = block.forward(residual[:20].clone(), attn[:20], k[:20])
    s.synchronize()
    b = block.forward(residual[:20].clone(), attn[:20], k[:20])
    assert block.device_status() == 0 and torch.equal(a, b)
    with pytest.raises(ValueError):
        K.synthetic(T=8)[0].forward(residual, attn, k)


def test_balancing_evens_the_load():
    block, residual, attn, k, adapter = K.synthetic(T=512, seed=3)
    spread = []           # how far the heaviest expert is over the mean load
    for _ in range(150):
        block.forward(residual.clone(), attn, k, adapter)
        load = block.load.float()
        spread.append(float(load.max() / load.mean()) - 1.0)
        block.balance(0.002)
    assert block.device_status() == 0
    assert np.mean(spread[-20:]) < 0.8 * np.mean(spread[:5])


def test_block_in_a_cuda_graph():
    block, residual, attn, k, adapter = K.synthetic(T=32, seed=5)
    want = block.forward(residual.clone(), attn, k, adapter)
    work, g = residual.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block.forward(work, attn, k, adapter)
    work.copy_(residual)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and block.device_status() == 0
    assert B.moe_status_string(0) == "MOE_OK"
