"""moe_lora_project against the float64 form.

Tolerance of a value before the SwiGLU: fp32 sums of K + r products (their
order is free: K 2^-24 of the sum of the terms' sizes), the low-rank
intermediate as two bf16 (2^-17 of the adapter terms, 2^-16 allowed), and y
rounded to bf16 (2^-8 of the value).  SwiGLU: |d silu(g) u| <= 1.1 |u| dg + |silu(g)| du, with
dg, du the bounds above without the last rounding.
"""
import numpy as np
import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from oracle import lora as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _make(T, K, N, n, r, seed, ldx=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    v = dict(x=rnd(T, ldx or K).bfloat16()[:, :K], w=(rnd(N, K) * K ** -0.5).bfloat16(),
             a=(rnd(max(n, 1), r, K) * K ** -0.5).bfloat16(),
             b=(rnd(max(n, 1), N, r) * 0.5 * r ** -0.5).bfloat16())
    v["ranks"] = torch.randint(0, r + 1, (max(n, 1),), generator=g, device=DEV, dtype=torch.int32)
    v["scales"] = 0.5 + 1.5 * torch.rand(max(n, 1), generator=g, device=DEV)
    return v


def _np(t):
    return t.double().cpu().numpy()


def _call(v, adapter, swiglu=False, ldy=0, ldx=0, n=None):
    T, K = v["x"].shape
    N, r = v["w"].shape[0], v["a"].shape[1]
    outs = N // 2 if swiglu else N
    d = B.LoraDesc(T=T, K=K, N=N, n_adapters=v["a"].shape[0] if n is None else n, r_max=r,
                   swiglu=swiglu, ldx=ldx, ldy=ldy)
    y = torch.full((T, ldy or outs), 99.0, dtype=torch.bfloat16, device=DEV)[:, :outs]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.moe_lora_workspace_size(d), dtype=torch.uint8, device=DEV)
    B.check(B.moe_lora_project(d, v["x"], v["w"], v["a"], v["b"], v["ranks"], v["scales"], adapter,
                               y, st, ws))
    return y, B.moe_get_device_status(st)


def _check(v, adapter, swiglu=False, ldy=0, ldx=0, status=0, rows=None):
    T, K = v["x"].shape
    y, st = _call(v, torch.tensor(adapter, dtype=torch.int32, device=DEV), swiglu, ldy, ldx)
    assert st == status
    r = np.clip(v["ranks"].cpu().numpy(), 0, v["a"].shape[1])
    a, b = _np(v["a"]), _np(v["b"])
    ref, base, low = L.project(_np(v["x"]), _np(v["w"]), a, b, r, _np(v["scales"]),
                               np.asarray(adapter), False)
    err = (K + 160) * 2.0 ** -24 * base + 2.0 ** -16 * low
    if swiglu:
        n = ref.shape[1] // 2
        g, u = ref[:, :n], ref[:, n:]
        s = g / (1 + np.exp(-g))
        err = 1.1 * np.abs(u) * err[:, :n] + (np.abs(s) + err[:, :n]) * err[:, n:]
        ref = L.swiglu_of(ref)
    bad = ~(np.abs(_np(y) - ref) <= err + 2.0 ** -8 * np.abs(ref) + 1e-30)
    if rows is not None:
        bad = bad[rows]
    assert not bad.any(), np.argwhere(bad)[:5]
    return y


def _spread(T, n, seed, none=0.2, request=1):
    rng = np.random.default_rng(seed)
    a = rng.integers(0, n, (T + request - 1) // request)
    a[rng.random(len(a)) < none] = -1
    return np.repeat(a, request)[:T].astype(np.int32)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 600,
                               1030])
@pytest.mark.parametrize("swiglu", [False, True])
def test_token_counts(T, swiglu):
    _check(_make(T, 256, 384, 5, 16, T), _spread(T, 5, T), swiglu)


@pytest.mark.parametrize("K,N", [(8, 2), (64, 64), (72, 130), (264, 126), (520, 258), (1000, 70),
                                 (2048, 1024), (136, 1)])
@pytest.mark.parametrize("T", [3, 40, 300])
def test_widths(T, K, N):
    _check(_make(T, K, N, 4, 8, K + N), _spread(T, 4, K))
    if N % 2 == 0:
        _check(_make(T, K, N, 4, 8, K + N), _spread(T, 4, K), swiglu=True)


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("T", [1, 30, 150, 700])
def test_ranks(T, r):
    _check(_make(T, 256, 192, 6, r, r), _spread(T, 6, r, request=max(1, T // 9)))


@pytest.mark.parametrize("N,ldy", [(2048, 0), (2050, 0), (2049, 0), (2049, 2052), (2049, 2056)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_tokens_rows_at_any_alignment(N, ldy, swiglu):
    N = 2 * N if swiglu else N
    _check(_make(3001, 512, N, 5, 24, N + ldy), _spread(3001, 5, ldy, request=300), swiglu, ldy=ldy)


@pytest.mark.parametrize("T", [64, 256, 700])
def test_every_token_its_own_adapter(T):
    _check(_make(T, 128, 192, 300, 16, T), (np.arange(T) * 7 % 300).astype(np.int32))


@pytest.mark.parametrize("T", [5, 100, 300])
def test_one_adapter_none_and_no_pool(T):
    v = _make(T, 128, 192, 3, 16, T)
    v["ranks"][1] = 16
    _check(v, np.full(T, 1, np.int32))
    _check(v, np.full(T, -1, np.int32))
    y, st = _call(v, None, n=0)
    assert st == 0
    z, _ = _call(v, torch.full((T,), -1, dtype=torch.int32, device=DEV))
    assert torch.equal(y, z)
    v["ranks"][:] = 0
    z, _ = _call(v, torch.zeros(T, dtype=torch.int32, device=DEV))
    assert torch.equal(y, z)


@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("swiglu", [False, True])
def test_strides(T, swiglu):
    N = 200
    outs = N // 2 if swiglu else N
    for ldy in (outs + 1, outs + 24):
        y = _check(_make(T, 96, N, 4, 16, T, ldx=104), _spread(T, 4, T), swiglu, ldy=ldy, ldx=104)
        base = torch.as_strided(y, (T - 1, ldy), (ldy, 1))
        assert (base[:, outs:] == 99).all()


@pytest.mark.parametrize("T", [6, 100, 300])
def test_what_lies_past_the_ranks_is_not_used(T):
    v = _make(T, 128, 192, 4, 24, T)
    v["ranks"] = torch.tensor([0, 5, 16, 23], dtype=torch.int32, device=DEV)
    adapter = _spread(T, 4, T)
    clean = _check(v, adapter).clone()
    for i, r in enumerate([0, 5, 16, 23]):
        v["a"][i, r:] = float("nan")
        v["b"][i, :, r:] = float("inf")
    dirty, st = _call(v, torch.tensor(adapter, device=DEV))
    assert st == 0 and torch.equal(clean, dirty)


@pytest.mark.parametrize("T", [6, 100, 300])
def test_a_broken_adapter_stays_with_its_own_tokens(T):
    """One request's non-finite factors or activations change no other request."""
    v = _make(T, 128, 192, 4, 16, T)
    v["ranks"][:] = 16
    adapter = _spread(T, 4, T, none=0.3)
    adapter[:4] = [0, 1, 2, -1]
    clean, _ = _call(v, torch.tensor(adapter, device=DEV))
    for spoil in ("a", "b", "x"):
        w = {k: t.clone() for k, t in v.items()}
        if spoil == "x":
            w["x"][2] = float("nan")
            mine = np.arange(T) == 2
        else:
            w[spoil][2, 3, 5] = float("inf")
            w[spoil][2, 4, 1] = float("nan")
            mine = adapter == 2
        y, _ = _call(w, torch.tensor(adapter, device=DEV))
        other = torch.tensor(~mine, device=DEV)
        assert torch.equal(y[other], clean[other]), spoil


def test_indexes_and_ranks_out_of_range_are_reported_and_unused():
    for T in (9, 300):
        v = _make(T, 128, 64, 3, 8, T)
        adapter = _spread(T, 3, T)
        adapter[4] = 3
        adapter[5] = -2
        clean = adapter.copy()
        clean[4:6] = -1
        y, st = _call(v, torch.tensor(adapter, device=DEV))
        assert st == 8
        z, st = _call(v, torch.tensor(clean, device=DEV))
        assert st == 0 and torch.equal(y, z)
        v["ranks"] = torch.tensor([8, 9, -1], dtype=torch.int32, device=DEV)
        y, st = _call(v, torch.tensor(clean, device=DEV))
        assert st == 8
        clean[clean > 0] = -1
        z, _ = _call(v, torch.tensor(clean, device=DEV))
        assert torch.equal(y, z)


def test_large_prefill_and_repeat_on_another_stream():
    T = 2500
    v = _make(T, 512, 640, 6, 32, 77)
    adapter = _spread(T, 6, 5, none=0.1, request=300)
    y = _check(v, adapter)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z, _ = _call(v, torch.tensor(adapter, device=DEV))
    assert torch.equal(y, z)
