"""Cases, plain forms and 64-bit forms of the operators around the MoE layer.

Three operators: group-limited routing with a balance bias (and the gradient of
its weights), the fused norms of a residual block (and their gradients), and a
projection shared by many requests with one low-rank adapter each.

``own`` selects what ``run`` calls: the plain torch form (float32 throughout,
rounded once at the end) or the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------- the cases

def _route(T, E, groups, kept, best, k, score, renorm, back=False, masked=0.0, **kw):
    return dict(op="route", T=T, E=E, groups=groups, kept=kept, best=best, k=k, score=score,
                renorm=renorm, back=back, masked=masked, **kw)


def _norm(T, H, res, act, gate, post, pre, back=False, offset=0.0, **kw):
    return dict(op="norm", T=T, H=H, res=res, act=act, gate=gate, post=post, pre=pre, back=back,
                offset=offset, **kw)


def _lora(T, K, N, adapters, rank, request, none=0.0, swiglu=False, **kw):
    return dict(op="lora", T=T, K=K, N=N, adapters=adapters, rank=rank, request=request, none=none,
                swiglu=swiglu, **kw)


def listed():
    return [
        # one token of a chat: 256 experts in 8 groups, sigmoid scores; pure latency
        _route(1, 256, 8, 4, 2, 8, "sigmoid", True, name="route one token"),
        # a prefill of 32 requests of 512 tokens on the same router
        _route(16384, 256, 8, 4, 2, 8, "sigmoid", True, name="route prefill 16384"),
        # softmax router without groups, per-token budgets, experts taken out of service, odd count
        _route(1777, 128, 1, 1, 1, 16, "softmax", False, masked=0.05, name="route softmax odd"),
        # training step: gradient of the gates of a softmax router (dense in the logits)
        _route(16384, 128, 8, 3, 1, 8, "softmax", False, back=True, name="route backward softmax"),
        # one decode token through post-norm, residual and the next pre-norm
        _norm(1, 7168, "bf16", "bf16", "none", True, True, name="norm one token"),
        # the same for a 16384-token prefill
        _norm(16384, 7168, "bf16", "bf16", "none", True, True, name="norm prefill 16384"),
        # float32 residual stream, a gate per channel, an odd hidden size and token count
        _norm(1023, 1001, "f32", "bf16", "channel", True, True, offset=1.0, name="norm odd f32"),
        # training step: gradients of the whole fused step with a gate per token
        _norm(8192, 2048, "bf16", "bf16", "token", True, True, back=True, name="norm backward"),
        # one decode token with an adapter on the shared expert's gate|up projection
        _lora(1, 7168, 4096, 8, 16, 1, name="lora one token"),
        # 64 requests of one token, up to 48 adapters of mixed ranks, some requests without one
        _lora(64, 7168, 4096, 48, 32, 1, none=0.1, name="lora decode 64"),
        # ragged mixture of short prompts, odd widths, SwiGLU of the shared expert
        _lora(777, 2056, 1538, 9, 24, 100, none=0.2, swiglu=True, name="lora ragged swiglu"),
        # a prefill of 32 requests of 512 tokens, an adapter each
        _lora(16384, 7168, 4096, 32, 64, 512, name="lora prefill 16384"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step from lo * step to hi * step, spread over its logarithm, odd multiples
    among them."""
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return step * (n + 1 if n * step == 3072 else n)


def draw(rng):
    op = rng.choice(["route", "norm", "lora"])
    if op == "route":
        groups, size = rng.choice([(1, 8), (1, 60), (1, 128), (1, 256), (2, 16), (4, 16), (4, 33),
                                   (8, 16), (8, 20), (8, 32), (16, 16), (32, 8), (64, 1), (128, 2)])
        kept = rng.randint((groups + 3) // 4, groups)
        k = rng.randint(1, min(16, kept * size))
        best = rng.choice([1, 2])
        return _route(_log(rng, 1, 16384), groups * size, groups, kept, best, k,
                      rng.choice(["sigmoid", "softmax"]), rng.random() < 0.5,
                      back=rng.random() < 0.4, masked=rng.choice([0.0, 0.0, 0.1]))
    if op == "norm":
        T, H = _log(rng, 1, 16384), rng.choice([_log(rng, 64, 8000), 64 * rng.randint(1, 40)])
        res, act = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        post, pre = rng.choice([(True, True), (True, False), (False, True)])
        return _norm(T, H, res, act, rng.choice(["none", "channel", "token", "full"]), post, pre,
                     back=rng.random() < 0.4, offset=rng.choice([0.0, 1.0]))
    swiglu = rng.random() < 0.3
    T = _log(rng, 1, 8192)
    return _lora(T, _log(rng, 16, 896, 8), _log(rng, 32, 2048, 2), _log(rng, 1, 64),
                 8 * rng.randint(1, 8), rng.choice([1, 1 + T // 8, 512]),
                 none=rng.choice([0.0, 0.2]), swiglu=swiglu)


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _choice64(logits, bias, c):
    """float64 scores s, biased scores with excluded units at -inf, and the least difference that
    any decision of the selection hangs on (all per token)."""
    l = logits.double()
    T, E = l.shape
    live = l > -math.inf
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, dim=1)
    b = torch.where(live, s + bias.double(), torch.tensor(-math.inf, dtype=l.dtype, device=DEV))
    per = b.view(T, c["groups"], E // c["groups"])
    best = torch.sort(per, dim=2, descending=True)[0][:, :, :c["best"]]
    rank = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
    rank = torch.where(best[:, :, 0] > -math.inf, rank, torch.full_like(rank, -math.inf))
    gs, gi = torch.sort(rank, dim=1, descending=True, stable=True)
    keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV).scatter_(
        1, gi[:, :c["kept"]], True)
    b = torch.where(keep[:, :, None].expand_as(per), per,
                    torch.full_like(per, -math.inf)).reshape(T, E)
    top = torch.sort(b, dim=1, descending=True, stable=True)
    gap = torch.full((T,), math.inf, dtype=l.dtype, device=DEV)
    if c["kept"] < c["groups"]:
        gap = torch.minimum(gap, (gs[:, c["kept"] - 1] - gs[:, c["kept"]]).nan_to_num(nan=math.inf))
    n = min(E, c["k"] + 1)
    if n > 1:
        d = (top[0][:, :n - 1] - top[0][:, 1:n]).nan_to_num(nan=math.inf)
        gap = torch.minimum(gap, d.min(1)[0])
    return s, top, gap


def _prepare_route(c, g):
    T, E = c["T"], c["E"]
    # token-dependent part plus a popularity that every token shares, as trained routers show
    logits = _randn(g, T, E) + 0.5 * _randn(g, 1, E)
    # the bias moves in steps of 0.001 towards balance
    bias = torch.round(_randn(g, E, std=20.0)) * 0.001
    if c["masked"]:
        off = torch.rand(E, generator=g, device=DEV) < c["masked"]
        logits[:, off] = -math.inf
    k = torch.randint((c["k"] + 1) // 2, c["k"] + 1, (T,), generator=g, device=DEV,
                      dtype=torch.int32)
    # Where two scores differ by less than their rounding, which one wins says nothing about the
    # operator: such tokens take the next decided token's logits.
    s, _, gap = _choice64(logits, bias, c)
    fine = gap > 4e-6 * (s.max(1)[0] + bias.abs().max())
    at = torch.where(fine, torch.arange(T, device=DEV), torch.full((T,), T, device=DEV))
    at = torch.flip(torch.cummin(torch.flip(at, [0]), 0)[0], [0])
    first = at[0].clamp(max=T - 1)
    logits = logits[torch.where(at < T, at, first)].contiguous()
    s = dict(logits=logits, bias=bias, k=k)
    if c["back"]:
        idx = _choice64(logits, bias, c)[1][1][:, :c["k"]].to(torch.int32)
        idx = torch.where(torch.arange(c["k"], device=DEV) < k[:, None], idx, -1)
        live = torch.gather(logits, 1, idx.clamp(min=0).long()) > -math.inf
        s["idx"] = torch.where(live, idx, -1).contiguous()
        s["d_w"] = _randn(g, T, c["k"])
    return s


def _prepare_norm(c, g):
    T, H, res, act = c["T"], c["H"], TYPES[c["res"]], TYPES[c["act"]]
    s = dict(r=_randn(g, T, H, std=2.0, dtype=res), y=_randn(g, T, H, std=0.7, dtype=act))
    mid = 1.0 - c["offset"]
    s["w_post"] = (mid + _randn(g, H, std=0.1)).to(act) if c["post"] else None
    s["w_pre"] = (mid + _randn(g, H, std=0.1)).to(act) if c["pre"] else None
    shape = {"none": None, "channel": (H,), "token": (T,), "full": (T, H)}[c["gate"]]
    s["gate"] = None if shape is None else _randn(g, *shape, std=0.5, dtype=act)
    if c["back"]:
        s["d_r"] = _randn(g, T, H, dtype=res)
        s["d_h"] = _randn(g, T, H, dtype=act) if c["pre"] else None
    return s


def _prepare_lora(c, g):
    T, K, N, n, r = c["T"], c["K"], c["N"], c["adapters"], c["rank"]
    s = dict(x=_randn(g, T, K, dtype=BF16), w=_randn(g, N, K, std=K ** -0.5, dtype=BF16),
             a=_randn(g, n, r, K, std=K ** -0.5, dtype=BF16),
             b=_randn(g, n, N, r, std=0.5 * r ** -0.5, dtype=BF16))
    # an adapter has any rank up to the pool's, and a scale of alpha / rank
    s["ranks"] = torch.randint((r + 1) // 2, r + 1, (n,), generator=g, device=DEV,
                               dtype=torch.int32)
    s["scales"] = 0.5 + 1.5 * torch.rand(n, generator=g, device=DEV)
    per = torch.randint(0, n, ((T + c["request"] - 1) // c["request"],), generator=g, device=DEV,
                        dtype=torch.int32)
    per = torch.where(torch.rand(per.shape, generator=g, device=DEV) < c["none"],
                      torch.full_like(per, -1), per)
    s["adapter"] = per.repeat_interleave(c["request"])[:T].contiguous()
    return s


def prepare(case, seed):
    g = _gen(seed)
    state = {"route": _prepare_route, "norm": _prepare_norm, "lora": _prepare_lora}[case["op"]](
        case, g)
    state["case"] = case
    if own:   # the descriptor, the workspace and the output buffers that a serving loop keeps
        state["handle"] = {"route": _handle_route, "norm": _handle_norm,
                           "lora": _handle_lora}[case["op"]](case, state)
    return state


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "norm": _own_norm, "lora": _own_lora}[op](state)
    back = state["case"].get("back")
    return {"route": _plain_route_back if back else _plain_route,
            "norm": _plain_norm_back if back else _plain_norm, "lora": _plain_lora}[op](state)


# ---------------------------------------------------------------- the plain forms

def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.max(dim=1, keepdim=True)[0])
    return e / e.sum(dim=1, keepdim=True)


def _plain_route(state):
    c, l = state["case"], state["logits"]
    T, E = l.shape
    s = _scores(l, c["score"])
    out = torch.full((), -math.inf, device=DEV)
    b = torch.where(l > -math.inf, s + state["bias"], out)
    per = b.view(T, c["groups"], E // c["groups"])
    best = torch.sort(per, dim=2, descending=True)[0][:, :, :c["best"]]
    rank = torch.where(best[:, :, 0] > -math.inf,
                       torch.where(best > -math.inf, best, torch.zeros((), device=DEV)).sum(2), out)
    kept = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :c["kept"]]
    keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV).scatter_(1, kept, True)
    b = torch.where(keep[:, :, None], per, out).reshape(T, E)
    top, idx = torch.sort(b, dim=1, descending=True, stable=True)
    top, idx = top[:, :c["k"]], idx[:, :c["k"]]
    live = (torch.arange(c["k"], device=DEV) < state["k"][:, None]) & (top > -math.inf)
    w = torch.where(live, torch.gather(s, 1, idx), torch.zeros((), device=DEV))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros((), device=DEV))
    load = torch.zeros(E, dtype=torch.int32, device=DEV).scatter_add_(
        0, idx.reshape(-1), live.reshape(-1).to(torch.int32))
    return {"idx": torch.where(live, idx, -1).to(torch.int32), "w": w * 2.5, "load": load}


def _plain_route_back(state):
    c, l, idx = state["case"], state["logits"], state["idx"]
    s = _scores(l, c["score"])
    at, live = idx.clamp(min=0).long(), idx >= 0
    zero = torch.zeros((), device=DEV)
    sel = torch.where(live, torch.gather(s, 1, at), zero)
    d = torch.where(live, state["d_w"], zero) * 2.5
    if c["renorm"]:
        total = sel.sum(1, keepdim=True)
        w = torch.where(total > 0, sel / total, zero)
        d = torch.where(live & (total > 0), (d - (d * w).sum(1, keepdim=True)) / total, zero)
    ds = torch.zeros_like(s).scatter_add_(1, at, d)
    if c["score"] == "sigmoid":
        return s * (1.0 - s) * ds
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _rms(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + 1e-6)


def _parts(state):
    """float32 residual, branch, gate ([T, H], [T, 1], [H] or 1) and the weights."""
    c = state["case"]
    gate = 1.0 if state["gate"] is None else state["gate"].float()
    if c["gate"] == "token":
        gate = gate[:, None]
    w = [None if state[n] is None else state[n].float() + c["offset"] for n in ("w_post", "w_pre")]
    return state["r"].float(), state["y"].float(), gate, w[0], w[1]


def _plain_norm(state):
    r, y, gate, w_post, w_pre = _parts(state)
    z = y if w_post is None else y * _rms(y) * w_post
    out = 0.9 * r + 1.25 * gate * z
    got = {"residual": out.to(state["r"].dtype)}
    if w_pre is not None:
        got["normed"] = (out * _rms(out) * w_pre).to(state["y"].dtype)
    return got


def _plain_norm_back(state):
    c = state["case"]
    r, y, gate, w_post, w_pre = _parts(state)
    n = y if w_post is None else y * _rms(y)
    z = n if w_post is None else n * w_post
    out = 0.9 * r + 1.25 * gate * z
    d, got = state["d_r"].float(), {}
    if w_pre is not None:
        m, d_h = out * _rms(out), state["d_h"].float()
        got["d_w_pre"] = (d_h * m).sum(0)
        d_m = d_h * w_pre
        d = d + _rms(out) * (d_m - m * (d_m * m).mean(dim=1, keepdim=True))
    got["d_residual"] = (0.9 * d).to(state["r"].dtype)
    d_z = 1.25 * d
    if c["gate"] == "channel":
        got["d_gate"] = (d_z * z).sum(0)
    elif c["gate"] == "token":
        got["d_gate"] = (d_z * z).sum(1)
    elif c["gate"] == "full":
        got["d_gate"] = (d_z * z).to(state["y"].dtype)
    d_z = d_z * gate
    if w_post is not None:
        got["d_w_post"] = (d_z * n).sum(0)
        d_n = d_z * w_post
        d_z = _rms(y) * (d_n - n * (d_n * n).mean(dim=1, keepdim=True))
    got["d_branch"] = d_z.to(state["y"].dtype)
    return got


def _plain_lora(state):
    c, x = state["case"], state["x"].float()
    n, r = c["adapters"], c["rank"]
    y = x @ state["w"].float().t()
    # every token against every adapter's columns, the other adapters' set to zero
    v = (x @ state["a"].float().reshape(n * r, -1).t()).view(-1, n, r)
    live = torch.arange(r, device=DEV) < state["ranks"][:, None]
    mine = state["adapter"][:, None] == torch.arange(n, device=DEV)
    v = torch.where(mine[:, :, None] & live, v * state["scales"][:, None], torch.zeros((), device=DEV))
    y = y + v.view(-1, n * r) @ state["b"].float().permute(0, 2, 1).reshape(n * r, -1)
    if c["swiglu"]:
        a, u = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = a / (1.0 + torch.exp(-a)) * u
    return y.to(BF16)


# ---------------------------------------------------------------- the library's calls

def _binding():
    from aware_moe_expert_gb300 import binding
    return binding


def _handle_route(c, s):
    B = _binding()
    T, E, k = c["T"], c["E"], c["k"]
    desc = B.LayerDesc(T=T, H=64, n_experts=E, n_sub=1, I_sub=64, k_max=k, score=c["score"],
                       renorm=c["renorm"], route_scale=2.5)
    groups = B.GroupRoute(n_groups=c["groups"], groups_kept=c["kept"], group_best=c["best"],
                          select_bias=s["bias"])
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    h = dict(B=B, desc=desc.c(), groups=groups.c(),
             status=torch.zeros(1, dtype=torch.int32, device=DEV))
    if c["back"]:
        h["d_logits"] = new(T, E, dtype=F32)
    else:
        h.update(idx=new(T, k, dtype=torch.int32), w=new(T, k, dtype=F32),
                 load=new(E, dtype=torch.int32))
    return h


def _own_route(state):
    h = state["handle"]
    B = h["B"]
    if state["case"]["back"]:
        B.check(B.moe_route_backward(h["desc"], state["logits"], state["idx"], state["d_w"],
                                     h["d_logits"], h["status"]))
        return h["d_logits"]
    B.check(B.moe_route_groups(h["desc"], h["groups"], None, None, state["logits"], state["k"],
                               None, h["idx"], h["w"], None, h["load"], h["status"], None))
    return {"idx": h["idx"], "w": h["w"], "load": h["load"]}


def _handle_norm(c, s):
    B = _binding()
    T, H, res, act = c["T"], c["H"], TYPES[c["res"]], TYPES[c["act"]]
    desc = B.BlockNormDesc(T=T, H=H, residual_dtype=res, act_dtype=act, gate=c["gate"], eps=1e-6,
                           weight_offset=c["offset"], residual_scale=0.9, branch_scale=1.25,
                           w_post=s["w_post"], w_pre=s["w_pre"])
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    h = dict(B=B, desc=desc.c())
    if not c["back"]:
        h["residual"] = new(T, H, dtype=res)
        if c["pre"]:
            h["normed"] = new(T, H, dtype=act)
        return h
    h["workspace"] = new(B.moe_block_norm_workspace_size(desc), dtype=torch.uint8)
    h["d_residual"], h["d_branch"] = new(T, H, dtype=res), new(T, H, dtype=act)
    if c["gate"] != "none":
        h["d_gate"] = (new(T, H, dtype=act) if c["gate"] == "full" else
                       new(H if c["gate"] == "channel" else T, dtype=F32))
    if c["post"]:
        h["d_w_post"] = new(H, dtype=F32)
    if c["pre"]:
        h["d_w_pre"] = new(H, dtype=F32)
    return h


def _own_norm(state):
    h = state["handle"]
    B, get = h["B"], h.get
    if not state["case"]["back"]:
        B.check(B.moe_block_norm(h["desc"], state["r"], state["y"], state["gate"], h["residual"],
                                 get("normed")))
        return {n: h[n] for n in ("residual", "normed") if n in h}
    B.check(B.moe_block_norm_backward(h["desc"], state["r"], state["y"], state["gate"],
                                      state["d_r"], state["d_h"], h["d_residual"], h["d_branch"],
                                      get("d_gate"), get("d_w_post"), get("d_w_pre"),
                                      h["workspace"]))
    return {n: h[n] for n in ("d_residual", "d_branch", "d_gate", "d_w_post", "d_w_pre") if n in h}


def _handle_lora(c, s):
    B = _binding()
    desc = B.LoraDesc(T=c["T"], K=c["K"], N=c["N"], n_adapters=c["adapters"], r_max=c["rank"],
                      swiglu=c["swiglu"])
    return dict(B=B, desc=desc.c(), status=torch.zeros(1, dtype=torch.int32, device=DEV),
                workspace=torch.empty(B.moe_lora_workspace_size(desc), dtype=torch.uint8,
                                      device=DEV),
                y=torch.empty(c["T"], c["N"] // 2 if c["swiglu"] else c["N"], dtype=BF16,
                              device=DEV))


def _own_lora(state):
    h = state["handle"]
    B = h["B"]
    B.check(B.moe_lora_project(h["desc"], state["x"], state["w"], state["a"], state["b"],
                               state["ranks"], state["scales"], state["adapter"], h["y"],
                               h["status"], h["workspace"]))
    return h["y"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        if not c["back"]:
            return {"bytes": 4.0 * T * E + 4 * E + 4 * T + 8.0 * T * k + 4 * E, "flops": 10.0 * T * E}
        dense = c["score"] == "softmax" and not c["renorm"]   # the other gradients need k logits
        return {"bytes": 4.0 * T * E + 8.0 * T * k + 4.0 * T * (E if dense else k),
                "flops": 10.0 * T * E}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        res, act = (2 if c["res"] == "bf16" else 4), (2 if c["act"] == "bf16" else 4)
        gate = {"none": 0, "channel": H, "token": T, "full": T * H}[c["gate"]]
        weights = H * (c["post"] + c["pre"])
        if not c["back"]:
            per = 2 * res + act * (1 + c["pre"])
            return {"bytes": float(T) * H * per + act * (gate + weights), "flops": 10.0 * T * H}
        per = 3 * res + act * (2 + c["pre"])
        d_gate = gate * act if c["gate"] == "full" else 4 * gate
        return {"bytes": float(T) * H * per + act * (gate + weights) + d_gate + 4 * weights,
                "flops": 25.0 * T * H}
    T, K, N, r = c["T"], c["K"], c["N"], c["rank"]
    requests = (T + c["request"] - 1) // c["request"] * (1.0 - c["none"])
    n = c["adapters"]
    active = n * (1.0 - (1.0 - 1.0 / n) ** requests)          # distinct adapters of random requests
    out = N // 2 if c["swiglu"] else N
    return {"bytes": 2.0 * (T * K + N * K + T * out) + 2.0 * active * 0.75 * r * (K + N) + 4.0 * T,
            "flops": 2.0 * T * K * N + 2.0 * T * (1.0 - c["none"]) * 0.75 * r * (K + N)}


# ---------------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] != "lora":
        return (_exact_route if c["op"] == "route" else _exact_norm)(c, s)
    if c["T"] * c["K"] * c["N"] > 6e11:
        return None
    x = s["x"].double()
    y = x @ s["w"].double().t()
    for a in range(c["adapters"]):   # adapter by adapter, on its own tokens
        rows, r = torch.nonzero(s["adapter"] == a).flatten(), int(s["ranks"][a])
        if rows.numel():
            v = float(s["scales"][a]) * (x[rows] @ s["a"][a, :r].double().t())
            y[rows] += v @ s["b"][a, :, :r].double().t()
    if c["swiglu"]:
        gate, up = y.chunk(2, dim=1)
        y = gate * torch.special.expit(gate) * up
    return y


def _exact_route(c, s):
    l = s["logits"].double()
    p = torch.special.expit(l) if c["score"] == "sigmoid" else torch.exp(
        l - torch.logsumexp(l, 1, keepdim=True))
    if c["back"]:
        # through automatic differentiation of the weights' definition
        l.requires_grad_(True)
        p = torch.special.expit(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
        live = s["idx"] >= 0
        w = torch.where(live, torch.gather(p, 1, s["idx"].clamp(min=0).long()), 0.0)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        (w * 2.5 * torch.where(live, s["d_w"].double(), 0.0)).sum().backward()
        return l.grad
    _, (top, order), _ = _choice64(s["logits"], s["bias"], c)
    k = c["k"]
    live = (torch.arange(k, device=DEV) < s["k"][:, None]) & (top[:, :k] > -math.inf)
    idx = torch.where(live, order[:, :k], -1)
    w = torch.where(live, torch.gather(p, 1, order[:, :k]), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    load = torch.bincount(idx[idx >= 0], minlength=c["E"])
    return {"idx": idx.to(torch.int32), "w": 2.5 * w, "load": load.to(torch.int32)}


def _exact_norm(c, s):
    leaf = {n: None if s[n] is None else s[n].double().requires_grad_(c["back"])
            for n in ("r", "y", "gate", "w_post", "w_pre")}
    H = c["H"]

    def norm(v, w):
        return v / torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / H + 1e-6) * (
            w + c["offset"])

    z = leaf["y"] if leaf["w_post"] is None else norm(leaf["y"], leaf["w_post"])
    gate = 1.0 if leaf["gate"] is None else leaf["gate"]
    if c["gate"] == "token":
        gate = gate.unsqueeze(1)
    out = 0.9 * leaf["r"] + 1.25 * gate * z
    h = None if leaf["w_pre"] is None else norm(out, leaf["w_pre"])
    if not c["back"]:
        return {"residual": out} if h is None else {"residual": out, "normed": h}
    loss = (out * s["d_r"].double()).sum()
    if h is not None:
        loss = loss + (h * s["d_h"].double()).sum()
    loss.backward()
    names = {"d_residual": "r", "d_branch": "y", "d_gate": "gate", "d_w_post": "w_post",
             "d_w_pre": "w_pre"}
    return {n: leaf[m].grad for n, m in names.items() if leaf[m] is not None}
