"""moe_lora_project where its own kernels' steps could go wrong."""
import numpy as np
import pytest
import torch
from test_gpu_lora import _check, _make, _spread
from test_gpu_lora_variants import plan

from aware_moe_expert_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,N", [(5, 64), (300, 256), (3000, 4096)])
def test_silu_of_large_gates(T, N):
    """Gates from -100 to 100, exact in the accumulators (one product each): SiLU within
    (4 + 1.2 |g|) 2^-23 of its value, y rounded once: y lies between
    the rounded ends of that interval; below -87 also 0."""
    K, outs = 64, N // 2
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(T)
    scale = 2.0 ** rng.integers(0, 3, T)
    x[:, 0] = torch.tensor(scale, device=DEV).bfloat16()
    x[:, 1] = 1
    w = torch.zeros(N, K, dtype=torch.bfloat16, device=DEV)
    w[:outs, 0] = torch.linspace(-25, 25, outs, device=DEV).bfloat16()
    w[outs:, 1] = (1 + torch.rand(outs, device=DEV)).bfloat16()
    d = B.LoraDesc(T=T, K=K, N=N, n_adapters=0, r_max=8, swiglu=True)
    y = torch.full((T, outs), 99.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.moe_lora_workspace_size(d), dtype=torch.uint8, device=DEV)
    B.check(B.moe_lora_project(d, x, w, None, None, None, None, None, y, st, ws))
    assert B.moe_get_device_status(st) == 0
    g = scale[:, None] * w[:outs, 0].double().cpu().numpy()
    u = w[outs:, 1].double().cpu().numpy()
    ref = g / (1 + np.exp(-g)) * u
    got = y.double().cpu().numpy()
    err = (4 + 1.2 * np.abs(g)) * 2.0 ** -23 * 1.01 * np.abs(ref)
    low, high = (torch.tensor(v).bfloat16().double().numpy() for v in (ref - err, ref + err))
    assert (((low <= got) & (got <= high)) | ((g < -87) & (got == 0))).all()
    assert (g < -87).any() and (g > 87).any()


@pytest.mark.parametrize("outs", [2041, 2042, 2047, 2048, 2049, 2050, 2055])
@pytest.mark.parametrize("swiglu", [False, True])
def test_columns_behind_the_outputs_keep_what_they_hold(outs, swiglu):
    """CTA pairs into rows that lie 16 bytes aligned apart: nothing behind their ends is
    written, whatever part of a 16-byte piece the last output leaves."""
    T, K, N, n, r = 3001, 64, 2 * outs if swiglu else outs, 5, 16
    assert plan(T, K, N, n, r, swiglu)[0] == 0
    for ldy in ((outs + 7) // 8 * 8, (outs + 7) // 8 * 8 + 8, outs + 1):
        v = _make(T, K, N, n, r, outs)
        y = _check(v, _spread(T, n, outs, request=300), swiglu, ldy=ldy)
        base = torch.as_strided(y, (T, ldy), (ldy, 1))
        assert (base[:, outs:] == 99).all()
