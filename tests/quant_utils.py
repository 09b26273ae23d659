"""Random 4-bit weights for the tests, packed by the library, and their float64 values."""
import numpy as np
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q

DEV = "cuda"


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def to64(t):
    return t.double().cpu().numpy()


def random_weights(rng, count, rows, K, kind, group, std=None):
    """(codes, scale bytes, factors): every code and scales over the whole of e4m3, zero and
    subnormal ones among them, most of them around 1."""
    codes = rng.integers(0, 256, (count, rows, K // 2), dtype=np.uint8)
    n = -(-K // group)
    scales = rng.integers(0x30, 0x44, (count, rows, n), dtype=np.uint8)
    odd = rng.random(scales.shape)
    scales = np.where(odd < 0.02, rng.integers(0, 8, scales.shape), scales)
    scales = np.where(odd > 0.995, 0x7E, scales).astype(np.uint8)
    std = K ** -0.5 / 4 if std is None else std
    return codes, scales, (std * (0.5 + rng.random(count))).astype(np.float32)


def pack(w, kind, group):
    codes, scales, factors = (torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in w)
    d = B.QuantDesc(codes.shape[0], codes.shape[1], 2 * codes.shape[2], kind, group)
    packed = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV)
    st = status()
    B.check(B.moe_quant_pack(d, codes, scales, factors, packed, st))
    assert B.moe_get_device_status(st) == 0
    return packed


class Layer:
    """Random experts (and a shared expert): packed, and in float64."""

    def __init__(self, seed, H, E, I, kind, group, shared=0):  # noqa: E741
        rng = np.random.default_rng(seed)
        self.H, self.E, self.I, self.shared, self.kind, self.group = H, E, I, shared, kind, group
        raw = {"gate_up": random_weights(rng, 2 * E, I, H, kind, group),
               "down": random_weights(rng, E, H, I, kind, group)}
        if shared:
            raw["shared_gate_up"] = random_weights(rng, 2, shared, H, kind, group)
            raw["shared_down"] = random_weights(rng, 1, H, shared, kind, group)
        self.w64 = {n: Q.weights(*w, kind, group) for n, w in raw.items()}
        self.packed = B.QuantWeights(kind, group, **{n: pack(w, kind, group) for n, w in raw.items()})

    def expert(self, e, x):
        return Q.ffn(x, self.w64["gate_up"][2 * e], self.w64["gate_up"][2 * e + 1], self.w64["down"][e])

    def shared_expert(self, x):
        return Q.ffn(x, self.w64["shared_gate_up"][0], self.w64["shared_gate_up"][1],
                     self.w64["shared_down"][0])


def within(got, y, dy, what=""):
    """got (bf16) is y rounded once, off by dy before that."""
    lim = Q.rounded(y, dy)
    off = np.abs(to64(got) - y)
    bad = ~(off <= lim)
    assert not bad.any(), (what, int(bad.sum()), float((off - lim)[bad].max()) if np.isfinite(off).all() else "nan",
                           np.argwhere(bad)[:4].tolist())
