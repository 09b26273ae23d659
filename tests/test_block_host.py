"""What the decoder block does on the host: its buffers, its checks, the streams
and arguments it hands to the library.  No GPU: the buffers are host memory, and
where a step runs, the library's calls are recorded instead of made."""
import dataclasses

import pytest
import torch

from aware_moe_expert_gb300 import binding as B
from aware_moe_expert_gb300 import block as K


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(B.LIB_PATH):
        from aware_moe_expert_gb300 import build
        build.build()
    return B.lib()


def _block(T=64, H=256, experts=32, I=128, k=6, shared=64, n_adapters=6, rank=16,  # noqa: E741
           groups=None):
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    w = K.BlockWeights(bf(H), bf(H), bf(H), bf(H), bf(experts, H), bf(experts, 2 * I, H),
                       bf(experts, H, I), bf(2 * shared, H), bf(H, shared), torch.zeros(experts))
    pool = K.Adapters(bf(n_adapters, rank, H), bf(n_adapters, 2 * shared, rank),
                      bf(n_adapters, rank, shared), bf(n_adapters, H, rank),
                      torch.full((n_adapters,), rank, dtype=torch.int32), torch.ones(n_adapters))
    layer = B.LayerDesc(T=T, H=H, n_experts=experts, n_sub=1, I_sub=I, k_max=k)
    return K.MoeBlock(layer, groups or B.GroupRoute(), w, pool, device="cpu")


@pytest.mark.parametrize("T,H,experts,I,k", [
    (342, 256, 32, 128, 6),      # a step of 341 tokens needs 8 MB more than one of 342
    (147, 2048, 64, 512, 8),
    (600, 128, 64, 64, 8), (1, 64, 8, 64, 2)])
def test_the_workspace_does_for_a_step_of_any_size(T, H, experts, I, k):  # noqa: E741
    block = _block(T, H, experts, I, k)
    for t in range(1, T + 1):
        d = dataclasses.replace(block.layer, T=t)
        assert B.moe_workspace_size(d) <= block.workspace.numel(), t
        for first in (True, False):
            assert B.moe_lora_workspace_size(block._lora(t, first)) <= block.lora_workspace.numel()


class _Calls:
    """Records the library's calls, and which stream is current, in their place."""

    def __init__(self, monkeypatch):
        self.current, self.calls = "current", []
        me = self

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                self.before, me.current = me.current, self.stream

            def __exit__(self, *_):
                me.current = self.before

        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
        for name in ("moe_block_norm", "moe_route_groups", "moe_permute", "moe_grouped_ffn",
                     "moe_lora_project", "moe_combine"):
            monkeypatch.setattr(B, name, self._fake(name))
        for name in ("empty_like", "sign"):
            monkeypatch.setattr(torch, name, self._through(name, getattr(torch, name)))

    def _on(self, stream):
        return self.current if stream is None else stream

    def _fake(self, name):
        def call(*args):
            params = getattr(B.lib(), name).argtypes
            stream = args[-1] if len(args) == len(params) else None
            self.calls.append((name, args, self._on(stream)))
            return 0
        return call

    def _through(self, name, real):
        def call(*args, **kw):
            self.calls.append((name, args, self.current))
            return real(*args, **kw)
        return call


def _step(T, H=256):
    return (torch.zeros(T, H), torch.zeros(T, H, dtype=torch.bfloat16),
            torch.ones(T, dtype=torch.int32), torch.zeros(T, dtype=torch.int32))


@pytest.mark.parametrize("stream,current", [(None, "current"), ("side", "side"),
                                            (4096, ("external", 4096))])
def test_a_step_and_its_balancing_are_work_of_one_stream(monkeypatch, stream, current):
    block, calls = _block(), _Calls(monkeypatch)
    block.forward(*_step(20), stream=stream)
    assert len(calls.calls) == 9         # eight of the library and the result's memory
    block.balance(0.01, stream=stream)
    names = [c[0] for c in calls.calls]
    assert names.count("empty_like") == 1 and names[-1] == "sign"
    assert [c[2] for c in calls.calls] == [current] * 10
    assert calls.current == "current"


def test_blocks_of_one_group_route_keep_their_own_bias(monkeypatch):
    groups = B.GroupRoute(n_groups=8, groups_kept=4, group_best=2)
    blocks = [_block(groups=groups) for _ in range(2)]
    assert groups.select_bias is None
    calls = _Calls(monkeypatch)
    for block in blocks:
        block.forward(*_step(5))
    used = [c[1][1].select_bias for c in calls.calls if c[0] == "moe_route_groups"]
    assert [b.data_ptr() for b in used] == [b.weights.select_bias.data_ptr() for b in blocks]
    assert used[0].data_ptr() != used[1].data_ptr()


@pytest.mark.parametrize("rank", [24, 128])
def test_a_pool_of_larger_rank_may_take_the_place_of_another(rank):
    for block in (_block(rank=16), _block(rank=8)):
        block.adapters = _block(rank=rank).adapters
        for first in (True, False):
            n = B.moe_lora_workspace_size(block._lora(block.layer.T, first))
            assert 0 < n <= block.lora_workspace.numel()


def test_a_replaced_selection_bias_is_the_one_that_routes(monkeypatch):
    block = _block()
    block.weights.select_bias = torch.ones(32)
    calls = _Calls(monkeypatch)
    block.forward(*_step(5))
    used = [c[1][1].select_bias for c in calls.calls if c[0] == "moe_route_groups"]
    assert used[0].data_ptr() == block.weights.select_bias.data_ptr()


def test_a_step_without_adapter_indexes_uses_no_pool(monkeypatch):
    block, calls = _block(), _Calls(monkeypatch)
    block.forward(*_step(5)[:3])
    used = [c[1] for c in calls.calls if c[0] == "moe_lora_project"]
    assert [a[0].n_adapters for a in used] == [0, 0]
    assert all(x is None for a in used for x in a[3:8])


@pytest.mark.parametrize("bad", [
    dict(attn=torch.zeros(20, 256)), dict(attn=torch.zeros(20, 128, dtype=torch.bfloat16)),
    dict(attn=torch.zeros(256, 20, dtype=torch.bfloat16).t()),
    dict(attn=torch.zeros(1, 256, dtype=torch.bfloat16).expand(20, 256)),
    dict(attn=torch.zeros(65, 256, dtype=torch.bfloat16)),
    dict(residual=torch.zeros(20, 256, dtype=torch.float16)), dict(residual=torch.zeros(19, 256)),
    dict(residual=torch.zeros(20, 512)[:, ::2]),
    dict(k=torch.ones(20, dtype=torch.int64)), dict(k=torch.ones(19, dtype=torch.int32)),
    dict(k=torch.ones(40, dtype=torch.int32)[::2]),
    dict(adapter=torch.ones(20, dtype=torch.int64)), dict(adapter=torch.ones(4, dtype=torch.int32))])
def test_a_step_refuses_what_the_library_would_misread(monkeypatch, bad):
    block, calls = _block(), _Calls(monkeypatch)
    step = dict(zip(("residual", "attn", "k", "adapter"), _step(20)))
    step.update(bad)
    with pytest.raises(ValueError):
        block.forward(*step.values())
    assert not calls.calls


def test_rows_at_a_stride_are_handed_on_with_it(monkeypatch):
    block, calls = _block(), _Calls(monkeypatch)
    _, _, k, adapter = _step(20)
    block.forward(torch.zeros(20, 300)[:, :256], torch.zeros(20, 264, dtype=torch.bfloat16)[:, :256],
                  k, adapter)
    first, last = [c[1][0] for c in calls.calls if c[0] == "moe_block_norm"]
    assert (first.ld_residual, first.ld_out, first.ld_branch) == (300, 300, 264)
    assert (last.ld_residual, last.ld_out, last.ld_branch) == (300, 300, 256)


def test_weights_and_pools_of_another_shape_are_refused():
    block = _block()
    for other in (_block(n_adapters=5), _block(shared=128)):
        pool = dataclasses.replace(block.adapters, down_a=other.adapters.down_a)
        with pytest.raises(ValueError):
            block.adapters = pool
    with pytest.raises(ValueError):
        block.adapters = dataclasses.replace(block.adapters, ranks=block.adapters.ranks.long())
    w = dataclasses.replace(block.weights, w_down=block.weights.w_down.transpose(1, 2))
    with pytest.raises(ValueError):
        K.MoeBlock(block.layer, B.GroupRoute(), w, device="cpu")
