"""4-bit weights whose bytes pass 2^32: experts of which the last lies behind it, in both
products, and one matrix longer than that.  The offsets are asserted."""
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from quant_utils import DEV, status

pytestmark = pytest.mark.gpu
I32 = torch.int32

# Every matrix the same codes but the last expert's: an offset cut to 32 bits reads another's.
H, I, E = 16384, 40960, 14  # noqa: E741
MATRIX = 128 * 320 * (8192 + 512)     # 128 x 320 tiles, either way round, of int4 and groups of 32
ROUNDINGS = 2.0 ** -8 * (2 / 3) ** 0.5
# One rounding of the activations to bf16 and one of the outputs: 2^-8 / sqrt(3) of the norm
# each at the most, and the first passes the second product as a relative change of its terms.


def _codes(g, count, rows, K):
    return torch.randint(0, 256, (count, rows, K // 2), dtype=torch.uint8, device=DEV, generator=g)


def _scales(*shape):
    return torch.full(shape, 0x38, dtype=torch.uint8, device=DEV)       # 1


def _pack(codes, factors):
    d = B.QuantDesc(codes.shape[0], codes.shape[1], 2 * codes.shape[2], "int4", 32)
    p, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
    B.check(B.moe_quant_pack(d, codes, _scales(*codes.shape[:2], d.K // 32), factors, p, st))
    assert B.moe_get_device_status(st) == 0
    return p


def _dense(codes, factor):
    """float64 of a matrix of codes."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double() - 8.0
    return q.mul_(float(factor))


def _off(y, want):
    return float((y.double() - want).norm() / want.norm())


@pytest.fixture(scope="module")
def experts():
    """(packed weights, the last expert's three matrices in float64)."""
    g = torch.Generator(device=DEV).manual_seed(1)
    raw = {}
    for name, per, rows, K in (("gate_up", 2, I, H), ("down", 1, H, I)):
        codes = _codes(g, 1, rows, K).expand(per * E, -1, -1).contiguous()
        codes[-per:] = _codes(g, per, rows, K)
        raw[name] = codes, torch.full((per * E,), K ** -0.5 / 4, device=DEV)
    weights = B.QuantWeights("int4", 32, *(_pack(*raw[n]) for n in ("gate_up", "down")))
    assert weights.gate_up.numel() // (2 * E) == MATRIX + 256 // (2 * E) and weights.down.numel() // E == MATRIX + 256 // E
    assert 2 * (E - 1) * MATRIX > 1 << 32 and (E - 1) * MATRIX > 1 << 32
    last = [_dense(raw["gate_up"][0][i], H ** -0.5 / 4) for i in (-2, -1)] + [_dense(raw["down"][0][-1], I ** -0.5 / 4)]
    yield weights, last
    del weights, last
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [2, 8, 40, 130])
def test_the_last_expert(experts, T):
    weights, (gate, up, down) = experts
    x = torch.randn(T, H, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).bfloat16()
    v = x.double() @ gate.t()
    want = (v / (1 + torch.exp(-v)) * (x.double() @ up.t())) @ down.t()
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=1)
    y, st = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), status()
    ws = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    offsets = torch.tensor([0] * E + [T], dtype=I32, device=DEV)
    B.check(B.moe_grouped_ffn_quant(d, weights, x, torch.arange(T, dtype=I32, device=DEV), offsets, y, st, ws))
    assert B.moe_get_device_status(st) == 0 and _off(y, want) <= ROUNDINGS
    # the layer: every token's router takes the last expert, with weight 1
    bias = torch.zeros(E, device=DEV)
    bias[-1] = 1
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=1, score="sigmoid", renorm=True, expert_bias=bias)
    ws = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    y.fill_(7.0)
    B.check(B.moe_layer_forward_quant(d, None, weights, x, torch.zeros(E, H, dtype=torch.bfloat16, device=DEV),
                                      torch.ones(T, dtype=I32, device=DEV), None, y, st, ws))
    assert B.moe_get_device_status(st) == 0 and _off(y, want) <= ROUNDINGS


@pytest.fixture(scope="module")
def matrix():
    N, K = 1 << 20, 8192
    codes = _codes(torch.Generator(device=DEV).manual_seed(2), 1, N, K)
    packed = _pack(codes, torch.full((1,), K ** -0.5 / 4, device=DEV))
    assert packed.numel() > 1 << 32
    yield codes[0], packed
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [1, 8, 9, 70])
def test_one_matrix(matrix, T):
    """Tiles from 2^32 bytes on start at row 986880: the rows from there, and the first ones."""
    codes, packed = matrix
    N, K = codes.shape[0], 2 * codes.shape[1]
    at = (1 << 32) // (K // 128 * 8704) * 128
    assert at + 4096 < N
    x = torch.randn(T, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(T)).bfloat16()
    y, st = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV), status()
    B.check(B.moe_quant_project(B.QuantProject(T, K, N, "int4", 32), x, packed, y, st,
                                torch.empty(256, dtype=torch.uint8, device=DEV)))
    assert B.moe_get_device_status(st) == 0
    for rows in (slice(0, 4096), slice(at - 256, at + 4096), slice(N - 4096, N)):
        assert _off(y[:, rows], x.double() @ _dense(codes[rows], K ** -0.5 / 4).t()) <= 2.0 ** -8 / 3 ** 0.5


def test_unpacking_one_matrix(matrix):
    codes, packed = matrix
    N, K = codes.shape[0], 2 * codes.shape[1]
    w = torch.full((1, N, K), 7.0, dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_unpack(B.QuantDesc(1, N, K, "int4", 32), packed, w))
    for r in range(0, N, 1 << 16):
        q = _dense(codes[r:r + (1 << 16)], K ** -0.5 / 4)
        # fp32, then bf16
        assert ((w[0, r:r + (1 << 16)].double() - q).abs() <= q.abs() * (2.0 ** -24 + 2.0 ** -8)).all()
