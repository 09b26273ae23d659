"""4-bit products where calls go wrong: empty and full experts, tokens without units,
bad indices, rows behind the last, values that are not finite, unaligned outputs,
captured and concurrent calls, weights written just before, matrices past 4 GB."""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import quant as Q
from quant_utils import DEV, Layer, pack, random_weights, status, to64, within

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _bf(rng, *shape):
    return torch.from_numpy(rng.normal(size=shape)).to(DEV, torch.bfloat16)


class _Call:
    """A layer call with its tensors, on a router that they are decided by."""

    def __init__(self, layer, T, k_max, seed=0, groups=None):
        rng = np.random.default_rng(seed)
        self.layer, self.groups = layer, groups
        self.x, self.router = _bf(rng, T, layer.H), _bf(rng, layer.E, layer.H) * layer.H ** -0.5
        self.k = torch.from_numpy(rng.integers(1, k_max + 1, T).astype(np.int32)).to(DEV)
        self.d = B.LayerDesc(T=T, H=layer.H, n_experts=layer.E, n_sub=1, I_sub=layer.I, k_max=k_max,
                             score="sigmoid", renorm=True, I_shared=layer.shared)
        self.ws = torch.empty(B.moe_quant_workspace_size(self.d), dtype=torch.uint8, device=DEV)
        self.st, self.out = status(), torch.full((T, layer.H), 7.0, dtype=torch.bfloat16, device=DEV)

    def run(self, stream=None):
        B.check(B.moe_layer_forward_quant(self.d, self.groups, self.layer.packed, self.x, self.router,
                                          self.k, None, self.out, self.st, self.ws, stream))
        return self.out

    def code(self):
        return B.moe_get_device_status(self.st)


@pytest.mark.parametrize("T", [1, 8, 9, 70])
def test_captured_and_replayed_on_new_inputs(T):
    layer = Layer(T, 256, 16, 128, "e2m1", 16, shared=64)
    c = _Call(layer, T, 5, seed=T)
    x2 = _bf(np.random.default_rng(99), T, 256)
    first = c.run().clone()
    assert torch.equal(c.run(), first)            # twice the same bits
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
        c.run()
    c.out.zero_()
    g.replay()
    assert torch.equal(c.out, first)
    c.x.copy_(x2)
    want = c.run().clone()
    c.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.out, want) and not torch.equal(want, first) and c.code() == 0


@pytest.mark.parametrize("T", [3, 40])
def test_two_calls_at_once_on_two_streams(T):
    layer = Layer(T, 512, 32, 192, "int4", 32, shared=128)
    calls = [_Call(layer, T, 6, seed=s) for s in (1, 2)]
    want = [c.run().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c.run(s)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c.out, w) and c.code() == 0


@pytest.mark.parametrize("T", [1, 2, 4])
def test_few_tokens_lose_their_outputs_rounding_only(T):
    """One expert of weight 1 and the shared one.  A rounding moves values by 2^-8 / sqrt(3) of
    them at the most in the mean square; activations rounded once to bf16 would double the square."""
    layer = Layer(T, 2048, 1, 512, "e2m1", 16, shared=256)
    c = _Call(layer, T, 1)
    x = to64(c.x)
    want = layer.expert(0, x)[0] + layer.shared_expert(x)[0]
    off = np.linalg.norm(to64(c.run()) - want) / np.linalg.norm(want)
    assert c.code() == 0 and off <= 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("T", [5, 20])
def test_tokens_without_units(T):
    """A bias of -inf takes every unit out: the shared expert alone, and the status says so."""
    layer = Layer(T, 192, 8, 64, "e2m1", 32, shared=64)
    none = B.GroupRoute(select_bias=torch.full((8,), float("-inf"), device=DEV))
    c = _Call(layer, T, 3, groups=none)
    out = c.run()
    assert c.code() == 7
    within(out, *layer.shared_expert(to64(c.x)))
    alone = Layer(T, 192, 8, 64, "e2m1", 32)
    c = _Call(alone, T, 3, groups=none)
    assert (c.run() == 0).all() and c.code() == 7


@pytest.mark.parametrize("T", [6, 30])
def test_budgets_out_of_range_are_reported(T):
    layer = Layer(T, 128, 8, 64, "int4", 16)
    c = _Call(layer, T, 3)
    want = c.run().clone()
    c.k[1] = 0
    out = c.run()
    assert c.code() == 7
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(out[rest], want[rest]) and (out[1] == 0).all()


@pytest.mark.parametrize("T", [1, 8, 9, 200])
def test_no_tokens_and_rows_behind_the_last(T):
    layer = Layer(3, 128, 4, 64, "e2m1", 16)
    c = _Call(layer, T, 2)
    out = torch.full((T + 2, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    c.out = out
    want = c.run().clone()
    assert (want[T:] == 7.0).all() and c.code() == 0
    c.d.T = 0
    c.run()
    assert torch.equal(out, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [4, 8, 16, 90])
def test_a_token_that_is_not_finite_keeps_to_itself(T, bad):
    rng = np.random.default_rng(T)
    for swiglu in (False, True):
        w = pack(random_weights(rng, 2 if swiglu else 1, 96, 264, "int4", 32), "int4", 32)
        d = B.QuantProject(T, 264, 192 if swiglu else 96, "int4", 32, swiglu)
        ws, st = torch.empty(B.moe_quant_project_workspace_size(d), dtype=torch.uint8, device=DEV), status()
        x = _bf(rng, T, 264)
        y = torch.empty(T, 96, dtype=torch.bfloat16, device=DEV)
        B.check(B.moe_quant_project(d, x, w, y, st, ws))
        x2, y2 = x.clone(), torch.empty_like(y)
        x2[2, 17] = bad
        B.check(B.moe_quant_project(d, x2, w, y2, st, ws))
        rest = [t for t in range(T) if t != 2]
        assert torch.equal(y[rest], y2[rest]) and not torch.isfinite(y2[2]).all()
        assert B.moe_get_device_status(st) == 0


@pytest.mark.parametrize("T", [2, 12, 70, 300])
@pytest.mark.parametrize("N,swiglu", [(130, False), (256, True), (33, False)])
def test_outputs_at_any_two_byte_address(T, N, swiglu):
    rng = np.random.default_rng(T + N)
    halves = 2 if swiglu else 1
    w = random_weights(rng, halves, N // halves, 136, "e2m1", 16)
    out, x, wp = N // halves, _bf(rng, T, 136), pack(w, "e2m1", 16)
    flat = torch.full((T * (out + 5) + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    for shift, ldy in ((1, 0), (3, out + 5), (0, out + 5)):
        flat.fill_(7.0)
        d = B.QuantProject(T, 136, N, "e2m1", 16, swiglu, 0, ldy)
        ld = ldy or out
        st, ws = status(), torch.empty(256, dtype=torch.uint8, device=DEV)
        B.check(B.moe_quant_project(d, x, wp, flat[shift:], st, ws))
        assert B.moe_get_device_status(st) == 0
        end = shift + (T - 1) * ld + out
        y = torch.as_strided(flat, (T, out), (ld, 1), shift)
        w64, x64 = Q.weights(*w, "e2m1", 16), to64(x)
        want = Q.swiglu(*Q.product(x64, w64[0]), *Q.product(x64, w64[1])) if swiglu else Q.product(x64, w64[0])
        within(y, *want)
        assert (flat[:shift] == 7.0).all() and (flat[end:] == 7.0).all()
        if ldy:
            gaps = torch.as_strided(flat, (T - 1, ld - out), (ld, 1), shift + out)
            assert (gaps == 7.0).all()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T,K,N", [(64, 1024, 4096), (65, 520, 700), (100, 640, 2048), (128, 264, 256), (129, 1160, 3584),
                                   (190, 1032, 1300), (300, 904, 1280), (321, 2056, 514), (1000, 136, 2050)])
def test_sums_split_over_clusters_of_every_width(T, K, N, swiglu):
    """Chunks of 64 tokens x blocks of outputs: from one item to more than a device holds."""
    rng = np.random.default_rng(T + N)
    halves = 2 if swiglu else 1
    kind, group = ("int4", 32) if T % 2 else ("e2m1", 16)
    w, x = random_weights(rng, halves, N // halves, K, kind, group), _bf(rng, T, K)
    d = B.QuantProject(T, K, N, kind, group, swiglu)
    st, ws = status(), torch.empty(256, dtype=torch.uint8, device=DEV)
    y = torch.full((T + 1, N // halves), 7.0, dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_project(d, x, pack(w, kind, group), y, st, ws))
    assert B.moe_get_device_status(st) == 0 and (y[T:] == 7.0).all()
    w64, x64 = Q.weights(*w, kind, group), to64(x)
    within(y[:T], *(Q.swiglu(*Q.product(x64, w64[0]), *Q.product(x64, w64[1])) if swiglu else Q.product(x64, w64[0])))


def _grouped(layer, T, k, token, offsets, rows=None):
    x = _bf(np.random.default_rng(5), T, layer.H)
    d = B.LayerDesc(T=T, H=layer.H, n_experts=layer.E, n_sub=1, I_sub=layer.I, k_max=k)
    y = torch.full((T * k, layer.H), 7.0, dtype=torch.bfloat16, device=DEV)
    st, ws = status(), torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    t = lambda v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    B.check(B.moe_grouped_ffn_quant(d, layer.packed, x, t(token), t(offsets), y, st, ws))
    return to64(x), y, B.moe_get_device_status(st)


@pytest.mark.parametrize("T,N", [(2300, 2100), (2300, 2304), (2432, 4096), (1300, 3585)])
def test_last_rounds_of_a_dense_product(T, N):
    """Some items more than SMs, with an odd number of row tiles and an even one."""
    rng = np.random.default_rng(N)
    w, x = random_weights(rng, 1, N, 72, "e2m1", 16), _bf(rng, T, 72)
    st, ws = status(), torch.empty(256, dtype=torch.uint8, device=DEV)
    y = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    B.check(B.moe_quant_project(B.QuantProject(T, 72, N, "e2m1", 16), x, pack(w, "e2m1", 16), y, st, ws))
    assert B.moe_get_device_status(st) == 0 and (y[T:] == 7.0).all()
    within(y[:T], *Q.product(to64(x), Q.weights(*w, "e2m1", 16)[0]))


@pytest.mark.parametrize("E", [17, 18])
def test_last_rounds_of_experts(E):
    """Nine blocks of outputs of 17 or 18 experts on 152 SMs, the last block of one tile."""
    layer = Layer(E, 2112, E, 64, "int4", 32)
    x, y, code = _grouped(layer, 3 * E, 1, list(range(3 * E)), list(range(0, 3 * E + 1, 3)))
    assert code == 0
    for e in range(E):
        within(y[3 * e:3 * e + 3], *layer.expert(e, x[3 * e:3 * e + 3]))
    c = _Call(layer, 100, 6, seed=E)            # fp32 rows between the products
    only, many = [], c.run().clone()
    for t0 in range(0, 100, 4):                 # the few-token kernels on the same tokens
        part = _Call(layer, 4, 6)
        part.x, part.router, part.k = c.x[t0:t0 + 4], c.router, c.k[t0:t0 + 4].contiguous()
        only.append(part.run().clone())
    few = torch.cat(only)
    assert c.code() == 0
    # both are within a rounding of the output and one of the activations of the same sums
    off = (many.double() - few.double()).norm() / few.double().norm()
    assert float(off) <= (2 + 1) ** 0.5 * 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("T", [3, 200])
def test_all_tokens_to_one_expert_and_none(T):
    layer = Layer(7, 128, 5, 64, "e2m1", 32)
    x, y, code = _grouped(layer, T, 2, list(range(T)), [0, 0, 0, T, T, T])
    assert code == 0 and (y[T:] == 7.0).all()
    within(y[:T], *layer.expert(2, x))
    _, y, code = _grouped(layer, T, 2, [0], [0] * 6)
    assert code == 0 and (y == 7.0).all()


def test_bad_indexes_are_reported():
    layer = Layer(7, 128, 3, 64, "int4", 16)
    T = 10
    token = list(range(T))
    for bad in (-1, T, 1 << 30):
        wrong = list(token)
        wrong[4] = bad
        x, y, code = _grouped(layer, T, 1, wrong, [0, 3, 3, T])
        assert code == 8
        within(y[:3], *layer.expert(0, x[:3]))
        rest = [3, 5, 6, 7, 8, 9]
        within(y[rest], *layer.expert(2, x[rest]))
        assert (y[4] == 0).all()                     # read as zeros
    for offsets in ([0, 3, 2, T], [0, 3, 3, T + 1], [-1, 3, 3, T], [0, 1 << 30, 1 << 30, 1 << 30]):
        _, y, code = _grouped(layer, T, 1, token, offsets)
        assert code == 8 and (y == 7.0).all()


@pytest.mark.parametrize("T", [1, 8, 60])
def test_weights_packed_by_the_launch_before(T):
    """No wait between packing and the product, over and over with other weights."""
    rng = np.random.default_rng(T)
    x, d = _bf(rng, T, 1024), B.QuantProject(T, 1024, 2048, "e2m1", 16)
    qd = B.QuantDesc(1, 2048, 1024, "e2m1", 16)
    ws, st = torch.empty(256, dtype=torch.uint8, device=DEV), status()
    sets = [[torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in random_weights(rng, 1, 2048, 1024, "e2m1", 16)]
            for _ in range(2)]
    want = []
    for s in sets:
        p, y = torch.empty(B.moe_quant_size(qd), dtype=torch.uint8, device=DEV), torch.empty(T, 2048, dtype=torch.bfloat16, device=DEV)
        B.check(B.moe_quant_pack(qd, *s, p, st))
        torch.cuda.synchronize()
        B.check(B.moe_quant_project(d, x, p, y, st, ws))
        want.append(y)
    p, got = torch.empty(B.moe_quant_size(qd), dtype=torch.uint8, device=DEV), []
    for i in range(40):
        y = torch.empty(T, 2048, dtype=torch.bfloat16, device=DEV)
        B.check(B.moe_quant_pack(qd, *sets[i % 2], p, st))
        B.check(B.moe_quant_project(d, x, p, y, st, ws))
        got.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(got))
    assert B.moe_get_device_status(st) == 0


@pytest.mark.parametrize("T", [2, 40, 130])
def test_matrices_past_four_gigabytes(T):
    """Three matrices of 1.4 GB as experts: the last one's rows lie past 2^32 bytes."""
    H, I, E = 16384, 78080, 2  # noqa: E741
    g = torch.Generator(device=DEV).manual_seed(1)
    def raw(count, rows, K):
        return (torch.randint(0, 256, (count, rows, K // 2), dtype=torch.uint8, device=DEV, generator=g),
                torch.full((count, rows, K // 32), 0x38, dtype=torch.uint8, device=DEV),
                torch.full((count,), K ** -0.5 / 4, device=DEV))

    def packed(w):
        d = B.QuantDesc(w[0].shape[0], w[0].shape[1], 2 * w[0].shape[2], "int4", 32)
        p, st = torch.empty(B.moe_quant_size(d), dtype=torch.uint8, device=DEV), status()
        B.check(B.moe_quant_pack(d, *w, p, st))
        assert B.moe_get_device_status(st) == 0
        return p

    def dense(w, i):
        c = w[0][i]
        q = torch.stack((c & 15, c >> 4), dim=-1).flatten(-2).double() - 8.0
        return q * float(w[2][i])

    gu, dn = raw(2 * E, I, H), raw(E, H, I)
    x = torch.randn(T, H, device=DEV, generator=g).bfloat16()
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=1)
    weights = B.QuantWeights("int4", 32, packed(gu), packed(dn))
    assert weights.gate_up.numel() > 1 << 32 or weights.gate_up.numel() > 2 ** 31
    ws, st = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV), status()
    y = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    token = torch.arange(T, dtype=I32, device=DEV)
    B.check(B.moe_grouped_ffn_quant(d, weights, x, token, torch.tensor([0, 0, T], dtype=I32, device=DEV), y, st, ws))
    assert B.moe_get_device_status(st) == 0
    gate = x.double() @ dense(gu, 2).t()
    a = gate / (1 + torch.exp(-gate)) * (x.double() @ dense(gu, 3).t())
    want = a @ dense(dn, 1).t()
    # one rounding of the activations and one of the outputs, over the norm
    assert float((y.double() - want).norm() / want.norm()) < 3e-3
    # the same through the layer call: the router takes the last expert for every token
    router = torch.zeros(E, H, dtype=torch.bfloat16, device=DEV)
    d = B.LayerDesc(T=T, H=H, n_experts=E, n_sub=1, I_sub=I, k_max=1, score="sigmoid", renorm=True,
                    expert_bias=torch.tensor([0.0, 1.0], device=DEV))
    ws = torch.empty(B.moe_quant_workspace_size(d), dtype=torch.uint8, device=DEV)
    k = torch.ones(T, dtype=I32, device=DEV)
    B.check(B.moe_layer_forward_quant(d, None, weights, x, router, k, None, y, st, ws))
    assert B.moe_get_device_status(st) == 0
    assert float((y.double() - want).norm() / want.norm()) < 3e-3
