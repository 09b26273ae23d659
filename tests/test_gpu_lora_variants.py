"""moe_lora_project in each of its kernels by name: tiles of 16 to 256 tokens, K whole
and split over a cluster, CTA pairs (tile 0), v by dot products and in tiles.

Which kernel serves a call is an estimate of the library's; the sizes here are
searched for with the library's own plan, so that a change of the estimate moves the
sizes and not what is covered.  Tolerances are those of tests/test_gpu_lora.py.
"""
import ctypes
import functools

import numpy as np
import pytest
import torch
from test_gpu_lora import _call, _check, _make, _spread

from aware_moe_expert_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = {name: code for code, name in B.STATUS_NAMES.items()}
NONFINITE, BAD_INDEX = CODES["MOE_ERR_NONFINITE"], CODES["MOE_ERR_BAD_INDEX"]


def plan(T, K, N, n, r, swiglu=False):
    """(tokens of a tile, 0: pairs; CTAs that split K; tokens of a tile of v, 0: dots)"""
    out = (ctypes.c_int32 * 3)()
    f = B.lib().moe_lora_plan
    f.argtypes = [ctypes.POINTER(B.MoeLoraDesc), ctypes.POINTER(ctypes.c_int32)]
    assert f(B.LoraDesc(T=T, K=K, N=N, n_adapters=n, r_max=r, swiglu=swiglu).c(), out) == 0
    return tuple(out)


@functools.lru_cache(maxsize=None)
def sizes(tile, split, n, r, swiglu=False):
    """The least (T, K, N) of a grid that the given kernel serves."""
    fits = [(T * K * N, T, K, N)
            for T in (12, 40, 70, 100, 130, 201, 300, 513, 700, 1030, 2001, 3001, 6001, 10001)
            for K in (136, 264, 520, 1040, 2056, 4104, 6472, 10008)
            for N in (130, 258, 514, 1030, 2050, 4098, 7030) if T * K * N < 6e10
            and plan(T, K, N, n, r, swiglu)[0] == tile
            and (plan(T, K, N, n, r, swiglu)[1] > 1) == split]
    assert fits, "no size of the grid is served by this kernel"
    return min(fits)[1:]


KERNELS = [(tile, split) for tile in (16, 32, 64, 128, 256) for split in (False, True)] + [(0, False)]


@pytest.mark.parametrize("tile,split", KERNELS)
@pytest.mark.parametrize("swiglu", [False, True])
def test_mixed_ranks_and_requests(tile, split, swiglu):
    """Forty adapters of rank 0 to 24, requests of one and of eleven tokens."""
    T, K, N = sizes(tile, split, 40, 24, swiglu)
    v = _make(T, K, N, 40, 24, T + K, ldx=K + 8)
    v["ranks"][:6] = torch.tensor([0, 1, 8, 16, 17, 24], dtype=torch.int32, device=DEV)
    for request in (1, 11):
        _check(v, _spread(T, 40, T, request=request), swiglu, ldx=K + 8)


@pytest.mark.parametrize("tile,split", KERNELS)
def test_an_adapter_for_every_token(tile, split):
    n = 64 if (tile, split) == (256, True) else 300      # with more, smaller tiles are taken
    T, K, N = sizes(tile, split, n, 16)
    _check(_make(T, K, N, n, 16, T), (np.arange(T) * 7 % n).astype(np.int32))


@pytest.mark.parametrize("tile,split", KERNELS)
def test_what_lies_past_the_ranks_is_not_used(tile, split):
    T, K, N = sizes(tile, split, 40, 24)
    v = _make(T, K, N, 40, 24, T)
    adapter = torch.tensor(_spread(T, 40, T), device=DEV)
    v["ranks"] = (torch.arange(40, dtype=torch.int32, device=DEV) * 5) % 25
    clean, st = _call(v, adapter)
    assert st == 0
    for i, r in enumerate(v["ranks"].tolist()):
        v["a"][i, r:] = float("nan")
        v["b"][i, :, r:] = float("inf") if i % 2 else float("nan")
    dirty, st = _call(v, adapter)
    assert st == 0 and torch.equal(clean, dirty)


@pytest.mark.parametrize("tile,split", KERNELS)
def test_a_broken_adapter_stays_with_its_own_tokens(tile, split):
    T, K, N = sizes(tile, split, 40, 24)
    v = _make(T, K, N, 40, 24, T)
    v["ranks"][:] = 24
    ids = _spread(T, 40, T, none=0.3)
    ids[:4] = [0, 1, 2, -1]
    adapter = torch.tensor(ids, device=DEV)
    clean, st = _call(v, adapter)
    assert st == 0
    for spoil in ("a", "b", "x"):
        w = {k: t.clone() for k, t in v.items()}
        if spoil == "x":
            w["x"][2] = float("nan")
            mine = np.arange(T) == 2
        else:
            w[spoil][2, 3, 5] = float("inf")
            w[spoil][2, 4, 17 if spoil == "b" else 1] = float("nan")
            mine = ids == 2
        y, st = _call(w, adapter)
        assert st == (NONFINITE if spoil == "b" else 0)
        assert torch.equal(y[torch.tensor(~mine, device=DEV)], clean[torch.tensor(~mine, device=DEV)])
        if spoil == "b":       # an element that is not finite counts as 0
            z = {k: t.clone() for k, t in v.items()}
            z["b"][2, 3, 5] = 0
            z["b"][2, 4, 17] = 0
            assert torch.equal(y, _call(z, adapter)[0])
        else:
            assert not torch.isfinite(y[2].float()).all()


@pytest.mark.parametrize("tile,split", KERNELS)
def test_indexes_and_ranks_out_of_range(tile, split):
    T, K, N = sizes(tile, split, 40, 24)
    v = _make(T, K, N, 40, 24, T)
    ids = _spread(T, 40, T)
    ids[4], ids[5], ids[6], ids[7] = 40, -2, 1, 2
    clean = ids.copy()
    clean[4:6] = -1
    y, st = _call(v, torch.tensor(ids, device=DEV))
    assert st == BAD_INDEX
    z, st = _call(v, torch.tensor(clean, device=DEV))
    assert st == 0 and torch.equal(y, z)
    v["ranks"][1], v["ranks"][2] = 25, -1
    y, st = _call(v, torch.tensor(clean, device=DEV))
    assert st == BAD_INDEX
    clean[(clean == 1) | (clean == 2)] = -1
    z, st = _call(v, torch.tensor(clean, device=DEV))
    assert st == 0 and torch.equal(y, z)


@pytest.mark.parametrize("tile,split", KERNELS)
def test_without_a_pool(tile, split):
    T, K, N = sizes(tile, split, 0, 8)
    v = _make(T, K, N, 0, 8, T)
    y, st = _call(v, None, n=0)
    x, w = v["x"].double().cpu().numpy(), v["w"].double().cpu().numpy()
    ref = x @ w.T
    err = K * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)
    assert st == 0
    assert (np.abs(y.double().cpu().numpy() - ref) <= err + 2.0 ** -8 * np.abs(ref) + 1e-30).all()


# r 128 and K as long as it takes for v to come from the tensor cores
@pytest.mark.parametrize("T,K,n,tile", [
    (16, 45000, 3, 16), (9, 81992, 2, 16), (32, 20008, 5, 32), (30, 22008, 5, 32), (64, 8008, 5, 64),
    (50, 11512, 9, 64), (128, 2056, 5, 128), (100, 4104, 3, 128), (300, 2056, 9, 256),
    (300, 136, 40, 256), (201, 4104, 40, 256), (1000, 520, 300, 256)])
def test_v_in_tiles(T, K, n, tile):
    assert plan(T, K, 66, n, 128)[2] == tile
    for request in (1, 7):
        _check(_make(T, K, 66, n, 128, T + n), _spread(T, n, T, request=request))


def test_v_in_tiles_of_broken_adapters():
    T, K, n = 201, 4104, 40
    assert plan(T, K, 66, n, 128)[2] == 256
    v = _make(T, K, 66, n, 128, 1)
    ids = _spread(T, n, 1)
    clean, _ = _call(v, torch.tensor(ids, device=DEV))
    v["a"][3] = float("nan")
    v["ranks"][3] = 128
    y, st = _call(v, torch.tensor(ids, device=DEV))
    keep = torch.tensor(ids != 3, device=DEV)
    assert st == 0 and (ids == 3).any() and torch.equal(y[keep], clean[keep])
