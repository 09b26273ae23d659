"""Calls on 4-bit weights where there is no device that can be used: a status, not the end
of the process.  In a process of its own that sees no device; no GPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLS = """
from aware_moe_expert_gb300 import binding as B
F, WS = 1 << 20, 1 << 21          # aligned, never dereferenced
d = B.LayerDesc(T={T}, H=256, n_experts=16, n_sub=1, I_sub=128, k_max=8, I_shared=64)
w = B.QuantWeights("{kind}", 16, F, F, F, F)
q = B.QuantDesc(2, 64, 64, "{kind}")
print(B.moe_quant_pack(q, F, F, F, F, F, 0), B.moe_quant_quantize(q, F, F, F, 0), B.moe_quant_unpack(q, F, F, 0),
      B.moe_quant_project(B.QuantProject({T}, 64, 128, "{kind}"), F, F, F, F, WS, 0),
      B.moe_quant_project(B.QuantProject({T}, 64, 128, "{kind}", swiglu=True), F, F, F, F, WS, 0),
      B.moe_layer_forward_quant(d, None, w, F, F, F, None, F, F, WS, 0),
      B.moe_layer_forward_quant(d, B.GroupRoute(), w, F, F, F, F, F, F, WS, 0),
      B.moe_grouped_ffn_quant(d, w, F, F, F, F, F, WS, 0), B.moe_shared_ffn_quant(d, w, F, F, F, WS, 0))
"""


@pytest.fixture(scope="module", autouse=True)
def lib():
    from aware_moe_expert_gb300 import binding as B
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()


@pytest.mark.parametrize("kind", ["e2m1", "int4"])
@pytest.mark.parametrize("T", [1, 8, 9, 64, 400])
def test_a_status_without_a_device(T, kind):
    r = subprocess.run([sys.executable, "-c", CALLS.format(T=T, kind=kind)], cwd=ROOT, capture_output=True, text=True,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-400:])
    assert r.stdout.split() == ["4"] * 9
