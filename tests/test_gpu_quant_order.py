"""Products right behind packing: they read weights before they wait, so packing has to end
with a launch that waits for it."""
import ctypes

import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from quant_utils import DEV, random_weights, status

pytestmark = pytest.mark.gpu


class _KernelNode(ctypes.Structure):          # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 6), ("shared", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p),
                ("ctx", ctypes.c_void_p)]


def _launches(call):
    """The names of the kernels of a captured call, in the order of their launches."""
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(stream)                                 # set-up that a capture does not allow
    torch.cuda.synchronize()
    cu, vp = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p

    def check(name, *args):
        assert getattr(cu, name)(*args) == 0, name

    graph, n = vp(), ctypes.c_size_t()
    check("cuStreamBeginCapture_v2", vp(stream.cuda_stream), 2)        # relaxed
    call(stream)
    check("cuStreamEndCapture", vp(stream.cuda_stream), ctypes.byref(graph))
    check("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (vp * n.value)()
    check("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    names = []
    for node in nodes:
        kind, name, k = ctypes.c_int(), ctypes.c_char_p(), _KernelNode()
        check("cuGraphNodeGetType", vp(node), ctypes.byref(kind))
        if kind.value == 0:
            check("cuGraphKernelNodeGetParams_v2", vp(node), ctypes.byref(k))
            if k.func:
                check("cuFuncGetName", ctypes.byref(name), vp(k.func))
            else:
                check("cuKernelGetName", ctypes.byref(name), vp(k.kern))
            names.append(name.value.decode())
    check("cuGraphDestroy", graph)
    return names


@pytest.mark.parametrize("quantize", [False, True])
def test_packing_ends_with_a_launch_that_waits(quantize):
    d = B.QuantDesc(2, 64, 128, "e2m1", 16)
    packed, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    if quantize:
        w = torch.randn(2, 64, 128, device=DEV).bfloat16()
        names = _launches(lambda s: B.check(B.moe_quant_quantize(d, w, packed, st, s)))
    else:
        raw = [torch.from_numpy(np.ascontiguousarray(v)).to(DEV)
               for v in random_weights(np.random.default_rng(0), 2, 64, 128, "e2m1", 16)]
        names = _launches(lambda s: B.check(B.moe_quant_pack(d, *raw, packed, st, s)))
    want = (["amax_kernel"] if quantize else []) + ["factor_kernel", "pack_kernel", "packed_kernel"]
    assert len(names) == len(want) and all(w in n for w, n in zip(want, names)), names


@pytest.mark.parametrize("T", [1, 8, 60])
def test_weights_quantized_by_the_launch_before(T):
    """No wait between quantising and the product, over and over with other weights."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, 1024, device=DEV, generator=g).bfloat16()
    d, qd = B.QuantProject(T, 1024, 2048, "int4", 32), B.QuantDesc(1, 2048, 1024, "int4", 32)
    ws, st = torch.empty(256, dtype=torch.uint8, device=DEV), status()
    sets = [(torch.randn(1, 2048, 1024, device=DEV, generator=g) / 32).bfloat16() for _ in range(2)]
    p = torch.empty(B.moe_quant_size(qd), dtype=torch.uint8, device=DEV)
    want = []
    for w in sets:
        y = torch.empty(T, 2048, dtype=torch.bfloat16, device=DEV)
        B.check(B.moe_quant_quantize(qd, w, p, st))
        torch.cuda.synchronize()
        B.check(B.moe_quant_project(d, x, p, y, st, ws))
        torch.cuda.synchronize()
        want.append(y)
    out = torch.empty(40, T, 2048, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    for i in range(40):
        B.check(B.moe_quant_quantize(qd, sets[i % 2], p, st))
        B.check(B.moe_quant_project(d, x, p, out[i], st, ws))
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(out))
    assert B.moe_get_device_status(st) == 0
