"""One feed-forward block of a decoder around the MoE layer, on one GPU.

    residual, h = norm(residual, attention output)    post-norm, residual, pre-norm
    routed      = group-limited routing of h, then the routed experts
    shared      = the shared expert, with the adapter of each token's request
    residual, h = norm(residual, routed + shared)     post-norm, residual, next pre-norm

Every step is a call of the library on the caller's stream; the block owns the
workspaces and the buffers between the steps.

``python -m aware_moe_expert_gb300.block`` runs a few steps of a small block on
synthetic inputs and balances its experts.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass, replace
from typing import Optional

import torch

from . import binding as B


@dataclass
class Adapters:
    """A pool of low-rank adapters beside the shared expert's two projections
    (A [n, r, in], B [n, out, r] bf16; ranks int32 [n]; scales fp32 [n])."""
    gate_up_a: torch.Tensor
    gate_up_b: torch.Tensor
    down_a: torch.Tensor
    down_b: torch.Tensor
    ranks: torch.Tensor
    scales: torch.Tensor


@dataclass
class BlockWeights:
    attn_post_norm: torch.Tensor          # [H]: norm of the attention output
    pre_norm: torch.Tensor                # [H]: norm of the block's input
    ffn_post_norm: torch.Tensor           # [H]: norm of the block's output
    next_pre_norm: torch.Tensor           # [H]: the next block's input norm
    router: torch.Tensor                  # [E_r, H]
    w_gate_up: torch.Tensor               # [E_r, 2 I, H]
    w_down: torch.Tensor                  # [E_r, H, I]
    shared_gate_up: torch.Tensor          # [2 I_shared, H]
    shared_down: torch.Tensor             # [H, I_shared]
    select_bias: torch.Tensor             # fp32 [E_r], moved by balance()


MAX_RANK = 128       # of a pool, the largest r_max


def _workspace_bytes(layer: B.LayerDesc) -> int:
    """Bytes of workspace that do for a step of any number of tokens up to layer.T.
    A step of fewer tokens can need more than one of layer.T does: it takes other
    kernels and splits its reductions further."""
    d, size = layer.c(), B.lib().moe_workspace_size
    n = 0
    for d.T in range(layer.T + 1):
        n = max(n, size(ctypes.byref(d)))
    if n == 0:
        raise B.MoeError(2, "moe_workspace_size")
    return n


def _on(stream):
    """The given stream (a torch stream or a handle) as the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _want(name, t, shape, dtypes, device, strided=False):
    """The library reads addresses: what is not this tensor is refused here."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.is_contiguous()
            and t.is_cuda == (device.type == "cuda")):
        return
    ok = (isinstance(t, torch.Tensor) and tuple(t.shape) == tuple(shape) and t.dtype in dtypes
          and t.device.type == device.type)
    if ok and strided:      # rows may lie apart
        ok = t.stride(-1) == 1 and (t.shape[0] < 2 or t.stride(0) >= t.shape[1])
    if not ok or not strided:
        kind = "rows" if strided else "contiguous"
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name}: {kind} {names} {list(shape)} on {device.type} wanted")


BF16, F32, I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


class MoeBlock:
    def __init__(self, layer: B.LayerDesc, groups: B.GroupRoute, weights: BlockWeights,
                 adapters: Optional[Adapters] = None, *, eps: float = 1e-6,
                 residual_scale: float = 1.0, branch_scale: float = 1.0, device="cuda"):
        """layer.T is the largest number of tokens of a step; layer.I_shared is
        taken from the weights (the shared expert runs here, with adapters)."""
        self.device = torch.device(device)
        self.layer, self.weights = layer, weights
        # this block's bias in a copy: blocks may be built from one GroupRoute
        self.groups = replace(groups, select_bias=weights.select_bias)
        self.eps, self.residual_scale, self.branch_scale = eps, residual_scale, branch_scale
        T, H, k = layer.T, layer.H, layer.k_max
        self.shared = weights.shared_down.shape[1]
        E, I = layer.E_r, layer.I_sub  # noqa: E741
        for name, shape in dict(attn_post_norm=(H,), pre_norm=(H,), ffn_post_norm=(H,),
                                next_pre_norm=(H,), router=(E, H), w_gate_up=(E, 2 * I, H),
                                w_down=(E, H, I), shared_gate_up=(2 * self.shared, H),
                                shared_down=(H, self.shared)).items():
            _want(name, getattr(weights, name), shape, BF16, self.device)
        self.adapters = adapters
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=self.device)  # noqa: E731
        i32 = torch.int32
        self.h, self.act, self.y_shared, self.y = new(T, H), new(T, self.shared), new(T, H), new(T, H)
        self.logits = new(T, layer.E_r, dtype=torch.float32)
        self.topk_idx, self.topk_w = new(T, k, dtype=i32), new(T, k, dtype=torch.float32)
        self.k_used, self.load = new(T, dtype=i32), new(layer.E_r, dtype=i32)
        self.counts, self.offsets = new(layer.E_r, dtype=i32), new(layer.E_r + 1, dtype=i32)
        self.sorted_token, self.inv_row = new(T * k, dtype=i32), new(T * k, dtype=i32)
        self.y_perm = new(T * k, H)
        self.status = torch.zeros(1, dtype=i32, device=self.device)
        self.workspace = new(_workspace_bytes(layer), dtype=torch.uint8)
        # for a pool of any rank: self.adapters may be replaced between steps
        n = min(B.moe_lora_workspace_size(replace(self._lora(T, first), r_max=MAX_RANK))
                for first in (True, False))
        if n == 0:
            raise B.MoeError(2, "moe_lora_workspace_size")
        self.lora_workspace = new(n, dtype=torch.uint8)

    @property
    def adapters(self) -> Optional[Adapters]:
        return self._adapters

    @adapters.setter
    def adapters(self, a: Optional[Adapters]):
        if a is not None:
            H, n = self.layer.H, a.ranks.shape[0]
            r, r2 = a.gate_up_a.shape[1], a.down_a.shape[1]
            for name, shape in dict(gate_up_a=(n, r, H), gate_up_b=(n, 2 * self.shared, r),
                                    down_a=(n, r2, self.shared), down_b=(n, H, r2)).items():
                _want(name, getattr(a, name), shape, BF16, self.device)
            _want("ranks", a.ranks, (n,), I32, self.device)
            _want("scales", a.scales, (n,), F32, self.device)
        self._adapters = a

    def _lora(self, T: int, first: bool, pool: bool = True) -> B.LoraDesc:
        a, H = self.adapters if pool else None, self.layer.H
        n, r = (0, 8) if a is None else a.gate_up_a.shape[:2] if first else a.down_a.shape[:2]
        if first:
            return B.LoraDesc(T=T, K=H, N=2 * self.shared, n_adapters=n, r_max=r, swiglu=True)
        return B.LoraDesc(T=T, K=self.shared, N=H, n_adapters=n, r_max=r)

    def _norm(self, residual, branch, w_post, w_pre, residual_out, normed):
        T, H = branch.shape
        ld, ld_branch = (residual.stride(0), branch.stride(0)) if T > 1 else (0, 0)
        d = B.BlockNormDesc(T=T, H=H, residual_dtype=residual.dtype, eps=self.eps,
                            ld_residual=ld, ld_out=ld, ld_branch=ld_branch,
                            residual_scale=self.residual_scale, branch_scale=self.branch_scale,
                            w_post=w_post, w_pre=w_pre, dev_status=self.status)
        B.check(B.moe_block_norm(d, residual, branch, None, residual_out, normed), "moe_block_norm")

    def forward(self, residual, attn, k_per_token, adapter_idx=None, stream=None):
        """residual (bf16 or fp32) and attn (bf16) [T, H], rows at any stride, budgets int32 [T],
        adapter_idx int32 [T] (-1: none; without it no token has one).  Updates residual in place and returns
        the next block's normed input; self.load has the assignments per unit.
        All of it is work of `stream` (default: the current one), on which the
        inputs have to be ready; the result belongs to that stream."""
        with _on(stream):
            return self._forward(residual, attn, k_per_token, adapter_idx)

    def _forward(self, residual, attn, k_per_token, adapter_idx):
        T, dev = attn.shape[0], self.device
        if T > self.layer.T:
            raise ValueError(f"{T} tokens, and buffers for {self.layer.T}")
        _want("attn", attn, (T, self.layer.H), BF16, dev, strided=True)
        _want("residual", residual, (T, self.layer.H), BF16 + F32, dev, strided=True)
        _want("k_per_token", k_per_token, (T,), I32, dev)
        if adapter_idx is not None:
            _want("adapter_idx", adapter_idx, (T,), I32, dev)
        _want("select_bias", self.weights.select_bias, (self.layer.E_r,), F32, dev)
        w, st, ws = self.weights, self.status, self.workspace
        a = None if adapter_idx is None else self.adapters
        self.groups.select_bias = w.select_bias      # which may have been replaced
        d = self.layer.c()
        d.T = T
        h = self.h[:T]
        self._norm(residual, attn, w.attn_post_norm, w.pre_norm, residual, h)
        idx, tw, k_used = self.topk_idx[:T], self.topk_w[:T], self.k_used[:T]
        B.check(B.moe_route_groups(d, self.groups, h, w.router, None, k_per_token,
                                   self.logits[:T], idx, tw, k_used, self.load, st, ws),
                "moe_route_groups")
        B.check(B.moe_permute(d, idx, k_used, self.counts, self.offsets, self.sorted_token,
                              self.inv_row, st, ws), "moe_permute")
        B.check(B.moe_grouped_ffn(d, h, self.sorted_token, self.offsets, w.w_gate_up, w.w_down,
                                  self.y_perm, st, ws), "moe_grouped_ffn")
        act, y_shared = self.act[:T], self.y_shared[:T]
        pool = lambda x, y: (x, y, a.ranks, a.scales, adapter_idx)  # noqa: E731
        none = (None,) * 5
        B.check(B.moe_lora_project(self._lora(T, True, a is not None), h, w.shared_gate_up,
                                   *(none if a is None else pool(a.gate_up_a, a.gate_up_b)), act,
                                   st, self.lora_workspace), "moe_lora_project")
        B.check(B.moe_lora_project(self._lora(T, False, a is not None), act, w.shared_down,
                                   *(none if a is None else pool(a.down_a, a.down_b)), y_shared,
                                   st, self.lora_workspace), "moe_lora_project")
        y = self.y[:T]
        B.check(B.moe_combine(d, self.y_perm, y_shared, self.inv_row, tw, k_used, y, st),
                "moe_combine")
        out = torch.empty_like(y)
        self._norm(residual, y, w.ffn_post_norm, w.next_pre_norm, residual, out)
        return out

    def balance(self, rate: float = 0.001, stream=None):
        """Moves the selection bias towards equal loads by `rate` a step, on the
        stream that the steps run on (default: the current one)."""
        with _on(stream):
            load = self.load.float()
            self.weights.select_bias += rate * torch.sign(load.mean() - load)

    def device_status(self, stream=None) -> int:
        return B.moe_get_device_status(self.status, stream)


def synthetic(T=64, H=256, experts=32, I=128, shared=256, n_adapters=6, rank=16, seed=0,  # noqa: E741
              device="cuda"):
    """A small block with random weights: (block, residual, attn, k, adapter_idx)."""
    g = torch.Generator(device=device).manual_seed(seed)
    bf = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=device) * std).bfloat16()  # noqa: E731
    norm = lambda: (1 + 0.1 * torch.randn(H, generator=g, device=device)).bfloat16()  # noqa: E731
    w = BlockWeights(norm(), norm(), norm(), norm(), bf(experts, H, std=H ** -0.5),
                     bf(experts, 2 * I, H, std=H ** -0.5), bf(experts, H, I, std=I ** -0.5),
                     bf(2 * shared, H, std=H ** -0.5), bf(H, shared, std=shared ** -0.5),
                     torch.zeros(experts, device=device))
    pool = Adapters(bf(n_adapters, rank, H, std=H ** -0.5),
                    bf(n_adapters, 2 * shared, rank, std=0.5 * rank ** -0.5),
                    bf(n_adapters, rank, shared, std=shared ** -0.5),
                    bf(n_adapters, H, rank, std=0.5 * rank ** -0.5),
                    torch.randint(rank // 2, rank + 1, (n_adapters,), generator=g, device=device,
                                  dtype=torch.int32),
                    0.5 + torch.rand(n_adapters, generator=g, device=device))
    layer = B.LayerDesc(T=T, H=H, n_experts=experts, n_sub=1, I_sub=I, k_max=6, score="sigmoid",
                        renorm=True, route_scale=2.5)
    block = MoeBlock(layer, B.GroupRoute(n_groups=8, groups_kept=4, group_best=2), w, pool,
                     device=device)
    k = torch.randint(3, 7, (T,), generator=g, device=device, dtype=torch.int32)
    adapter = torch.randint(-1, n_adapters, (T,), generator=g, device=device, dtype=torch.int32)
    return block, bf(T, H, std=2.0).float(), bf(T, H, std=0.5), k, adapter


def main():
    block, residual, attn, k, adapter = synthetic(T=512)
    for step in range(200):
        h = block.forward(residual.clone(), attn, k, adapter)
        load = block.load.float()
        if step % 50 == 0 or step == 199:
            print(f"step {step}: heaviest expert at {float(load.max() / load.mean()):.2f} of the "
                  f"mean load, |h| {float(h.float().abs().mean()):.3f}")
        block.balance()
    print("device status:", B.moe_status_string(block.device_status()))


if __name__ == "__main__":
    main()
