"""Cases, plain forms and 64-bit forms of the operators on 4-bit weights.

A weight matrix is 4-bit codes with a scale for every `group` consecutive inputs
of a row (e4m3) and one float32 factor:

    W[n, k] = factor * scale[n, k // group] * value(code[n, k])

where value() is e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) or the
integer code - 8.  Three operators: a projection, the whole MoE layer for few
tokens (routing, experts, shared expert, weighted sum), and the experts' FFN on
rows that a permutation has grouped by expert.

``own`` selects what ``run`` calls: the plain torch form (float32 throughout,
rounded once at the end) or the library's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
VALUES = {"e2m1": E2M1 + [-v for v in E2M1], "int4": [float(q - 8) for q in range(16)]}


# ---------------------------------------------------------------- the cases

def _project(T, K, N, code, group, swiglu=False, **kw):
    return dict(op="project", T=T, K=K, N=N, code=code, group=group, swiglu=swiglu, **kw)


def _layer(T, H, E, I, k, code, group, score="softmax", renorm=False, groups=0, kept=0, best=1,  # noqa: E741
           shared=0, **kw):
    return dict(op="layer", T=T, H=H, E=E, I=I, k=k, code=code, group=group, score=score,
                renorm=renorm, groups=groups, kept=kept, best=best, shared=shared, **kw)


def _experts(T, H, E, I, k, code, group, skew=0.0, **kw):  # noqa: E741
    return dict(op="experts", T=T, H=H, E=E, I=I, k=k, code=code, group=group, skew=skew, **kw)


def listed():
    return [
        # one token through a projection of a wide model: a chat with one user
        _project(1, 7168, 4096, "e2m1", 16, name="project one token"),
        # a few requests through the gate|up projection of a shared expert, odd widths
        _project(5, 2056, 1538, "int4", 32, swiglu=True, name="project five tokens odd"),
        # a decode batch of 64 requests
        _project(64, 7168, 4096, "e2m1", 32, name="project decode 64"),
        # a prefill of 32 requests of 512 tokens
        _project(16384, 7168, 4096, "e2m1", 16, name="project prefill 16384"),
        # one token through 256 sub-experts of 384, budgets up to 16: pure latency
        _layer(1, 2048, 256, 384, 16, "e2m1", 16, name="layer one token"),
        # eight requests on the same layer
        _layer(8, 2048, 256, 384, 16, "int4", 32, name="layer eight tokens"),
        # three requests, 256 experts in 8 groups behind a sigmoid router, and a shared expert
        _layer(3, 7168, 256, 2048, 8, "e2m1", 16, score="sigmoid", renorm=True, groups=8, kept=4,
               best=2, shared=2048, name="layer grouped and shared"),
        # a decode batch of 64 requests, 8 experts split in four
        _layer(64, 4096, 32, 3584, 8, "int4", 32, name="layer decode 64"),
        # ragged small model: widths that are no multiple of the tiles
        _experts(333, 320, 12, 192, 3, "int4", 16, skew=1.0, name="experts ragged"),
        # a decode batch of 1024 requests on 128 experts of 768
        _experts(1024, 2048, 128, 768, 8, "e2m1", 32, skew=0.5, name="experts 1024"),
        # a prefill of 16 requests of 512 tokens on them
        _experts(8192, 2048, 128, 768, 8, "e2m1", 16, skew=0.5, name="experts prefill 8192"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step from lo * step to hi * step, spread over its logarithm."""
    return step * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["project", "layer", "experts"])
    code, group = rng.choice(["e2m1", "int4"]), rng.choice([16, 32])
    if op == "project":
        return _project(_log(rng, 1, 8192), _log(rng, 2, 896, 8), _log(rng, 16, 2048, 2), code,
                        group, swiglu=rng.random() < 0.3)
    if op == "experts":
        E = _log(rng, 1, 256)
        return _experts(_log(rng, 1, 4096), _log(rng, 1, 32, 64), E, _log(rng, 1, 16, 64),
                        rng.randint(1, min(E, 8)), code, group, skew=rng.choice([0.0, 0.5, 1.0]))
    groups, size = rng.choice([(0, _log(rng, 4, 256)), (1, 60), (4, 16), (4, 33), (8, 32)])
    E = max(groups, 1) * size
    kept = rng.randint((groups + 1) // 2, groups) if groups else 0
    k = rng.randint(1, min(16, (kept or 1) * size))
    return _layer(_log(rng, 1, 256), _log(rng, 1, 64, 64), E, _log(rng, 1, 24, 64), k, code, group,
                  score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5,
                  groups=groups, kept=kept, best=rng.choice([1, 2]),
                  shared=rng.choice([0, 0, 64 * rng.randint(1, 16)]))


# ---------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape, std=1.0, dtype=F32):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _weights(g, count, rows, K, c):
    """Codes [count, rows, K / 2] (two a byte, the even input low), scales [count, rows, K / group]
    and factors [count] of weights that are normal with a standard deviation of K ** -0.5."""
    codes = torch.empty(count, rows, K // 2, dtype=torch.uint8, device=DEV)
    at = max(1, (1 << 26) // (rows * K))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    for i in range(0, count, at):
        v = _randn(g, min(at, count - i), rows, K)
        if c["code"] == "int4":     # a group's largest is near the last code
            q = torch.round(v * 2.8 + 8.0).clamp(0, 15).to(torch.uint8)
        else:
            q = torch.bucketize((v * 2.3).abs(), edges).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
        codes[i:i + at] = q[..., ::2] | q[..., 1::2] << 4
    groups = (K + c["group"] - 1) // c["group"]
    scales = (40.0 + 120.0 * torch.rand(count, rows, groups, generator=g, device=DEV)).to(
        torch.float8_e4m3fn)
    std = (2.8 if c["code"] == "int4" else 2.3) * 100.0 * K ** 0.5
    factor = (0.8 + 0.4 * torch.rand(count, generator=g, device=DEV)) / std
    return codes, scales, factor


def _choice64(logits, bias, c):
    """float64 scores s, what ranks the units (the logits, or scores with a bias under groups,
    units of dropped groups at -inf) sorted, and the least difference that a decision hangs on."""
    T, E = logits.shape
    s = torch.special.expit(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    b, gap = logits, torch.full((T,), math.inf, dtype=torch.float64, device=DEV)
    scale = 1.0
    if c["groups"]:
        b = s + bias.double()
        scale = s.max(1)[0] + bias.abs().max().double()
        per = b.view(T, c["groups"], E // c["groups"])
        rank = torch.sort(per, dim=2, descending=True)[0][:, :, :c["best"]].sum(2)
        gs, gi = torch.sort(rank, dim=1, descending=True, stable=True)
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV).scatter_(
            1, gi[:, :c["kept"]], True)
        b = torch.where(keep[:, :, None].expand_as(per), per,
                        torch.full_like(per, -math.inf)).reshape(T, E)
        if c["kept"] < c["groups"]:
            gap = gs[:, c["kept"] - 1] - gs[:, c["kept"]]
    top = torch.sort(b, dim=1, descending=True, stable=True)
    n = min(E, c["k"] + 1)
    if n > 1:
        d = (top[0][:, :n - 1] - top[0][:, 1:n]).nan_to_num(nan=math.inf)
        gap = torch.minimum(gap, d.min(1)[0])
    return s, top, gap / scale


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "project":
        halves = 2 if c["swiglu"] else 1
        s["x"] = _randn(g, c["T"], c["K"], dtype=BF16)
        s["w"] = _weights(g, halves, c["N"] // halves, c["K"], c)
    else:
        T, H, E, I, k = c["T"], c["H"], c["E"], c["I"], c["k"]  # noqa: E741
        s["x"] = _randn(g, T, H, dtype=BF16)
        s["gate_up"] = _weights(g, 2 * E, I, H, c)     # gate and up of an expert in turn
        s["down"] = _weights(g, E, H, I, c)
    if c["op"] == "experts":
        # every token takes k experts, some experts more often than others
        rank = torch.randperm(E, generator=g, device=DEV).to(F32)
        noise = torch.rand(T, E, generator=g, device=DEV)
        idx = torch.topk(torch.log(1.0 + rank) * -c["skew"] - torch.log(-torch.log(noise)), k,
                         dim=1)[1]
        unit, order = torch.sort(idx.reshape(-1), stable=True)
        s["token"] = torch.div(order, k, rounding_mode="floor").to(I32)
        s["offsets"] = torch.zeros(E + 1, dtype=I32, device=DEV)
        s["offsets"][1:] = torch.cumsum(torch.bincount(unit, minlength=E), 0)
    if c["op"] == "layer":
        s["k"] = torch.randint((k + 1) // 2, k + 1, (T,), generator=g, device=DEV, dtype=I32)
        s["router"] = _randn(g, E, H, std=H ** -0.5, dtype=BF16)
        s["bias"] = torch.round(_randn(g, E, std=20.0)) * 0.001 if c["groups"] else None
        if c["shared"]:
            s["shared_gate_up"] = _weights(g, 2, c["shared"], H, c)
            s["shared_down"] = _weights(g, 1, H, c["shared"], c)
        # Where two scores differ by less than the rounding of the logits, which one wins says
        # nothing about the operator: such tokens take the next decided token's inputs.
        fine = _choice64(s["x"].double() @ s["router"].double().t(), s["bias"], c)[2] > 2e-5
        at = torch.where(fine, torch.arange(T, device=DEV), torch.full((T,), T, device=DEV))
        at = torch.flip(torch.cummin(torch.flip(at, [0]), 0)[0], [0])
        s["x"] = s["x"][torch.where(at < T, at, at[0].clamp(max=T - 1))].contiguous()
    if own:   # the packed weights, descriptors, workspace and outputs that a serving loop keeps
        s["handle"] = _handle(c, s)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"project": _own_project, "layer": _own_layer, "experts": _own_experts}[op](state)
    return {"project": _plain_project, "layer": _plain_layer, "experts": _plain_experts}[op](state)


# ---------------------------------------------------------------- the plain forms

def _dense(w, c, units=None):
    """float32 matrices [count, rows, K], of the given units alone."""
    codes, scales, factor = w if units is None else [t[units] for t in w]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    value = torch.tensor(VALUES[c["code"]], device=DEV)[q.long()]
    s = scales.float() * factor[:, None, None]
    return value * s.repeat_interleave(c["group"], dim=2)[..., :q.shape[-1]]


def _swiglu(gate, up):
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_project(state):
    w = _dense(state["w"], state["case"])
    y = state["x"].float() @ w.flatten(0, 1).t()
    return (_swiglu(*y.chunk(2, dim=1)) if state["case"]["swiglu"] else y).to(BF16)


def _plain_rows(state, unit, token):
    """float32 outputs [rows, H] of rows sorted by unit; x row `token` of each."""
    c = state["case"]
    units, which, count = torch.unique_consecutive(unit, return_inverse=True, return_counts=True)
    place = torch.arange(unit.numel(), device=DEV) - (torch.cumsum(count, 0) - count)[which]
    x = torch.zeros(units.numel(), int(count.max()), c["H"], device=DEV)
    x[which, place] = state["x"].float()[token]
    pair = torch.stack((2 * units, 2 * units + 1), dim=1).flatten()
    w = _dense(state["gate_up"], c, pair).view(units.numel(), 2 * c["I"], c["H"])
    a = _swiglu(*torch.bmm(x, w.transpose(1, 2)).chunk(2, dim=2))
    return torch.bmm(a, _dense(state["down"], c, units).transpose(1, 2))[which, place]


def _plain_experts(state):
    n = state["offsets"][1:] - state["offsets"][:-1]
    unit = torch.arange(state["case"]["E"], device=DEV).repeat_interleave(n)
    return _plain_rows(state, unit, state["token"].long()).to(BF16)


def _plain_layer(state):
    c, x = state["case"], state["x"].float()
    l = x @ state["router"].float().t()
    T, E = l.shape
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.max(dim=1, keepdim=True)[0])
        s = e / e.sum(dim=1, keepdim=True)
    b = l
    if c["groups"]:
        b = (s + state["bias"]).view(T, c["groups"], -1)
        rank = torch.sort(b, dim=2, descending=True)[0][:, :, :c["best"]].sum(2)
        kept = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :c["kept"]]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        b = torch.where(keep[:, :, None], b, torch.full((), -math.inf, device=DEV)).view(T, E)
    idx = torch.sort(b, dim=1, descending=True, stable=True)[1][:, :c["k"]]
    live = torch.arange(c["k"], device=DEV) < state["k"][:, None]
    w = torch.where(live, torch.gather(s, 1, idx), torch.zeros((), device=DEV))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    token, slot = torch.nonzero(live, as_tuple=True)
    unit, order = torch.sort(idx[token, slot], stable=True)
    token, slot = token[order], slot[order]
    out = torch.zeros(T, c["H"], device=DEV)
    out.index_add_(0, token, _plain_rows(state, unit, token) * w[token, slot][:, None])
    if c["shared"]:
        y = x @ _dense(state["shared_gate_up"], c).flatten(0, 1).t()
        out = out + _swiglu(*y.chunk(2, dim=1)) @ _dense(state["shared_down"], c)[0].t()
    return out.to(BF16)


# ---------------------------------------------------------------- the library's calls

def _binding():
    from aware_moe_expert_gb300 import binding
    return binding


def _handle(c, s):
    B = _binding()
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731

    def pack(w):
        codes, scales, factor = w
        desc = B.QuantDesc(count=codes.shape[0], rows=codes.shape[1], K=2 * codes.shape[2],
                        code=c["code"], group=c["group"])
        packed = new(B.moe_quant_size(desc), dtype=torch.uint8)
        B.check(B.moe_quant_pack(desc, codes, scales, factor, packed, h["status"]))
        return packed

    h = dict(B=B, status=torch.zeros(1, dtype=I32, device=DEV))
    if c["op"] == "project":
        desc = B.QuantProject(T=c["T"], K=c["K"], N=c["N"], code=c["code"], group=c["group"],
                           swiglu=c["swiglu"])
        h.update(desc=desc.c(), w=pack(s["w"]),
                 y=new(c["T"], c["N"] // 2 if c["swiglu"] else c["N"], dtype=BF16),
                 workspace=new(B.moe_quant_project_workspace_size(desc), dtype=torch.uint8))
        return h
    layer = c["op"] == "layer"
    desc = B.LayerDesc(T=c["T"], H=c["H"], n_experts=c["E"], n_sub=1, I_sub=c["I"], k_max=c["k"],
                       score=c.get("score", "softmax"), renorm=c.get("renorm", False),
                       I_shared=c.get("shared", 0))
    shared = layer and c["shared"]
    h["weights"] = B.QuantWeights(code=c["code"], group=c["group"], gate_up=pack(s["gate_up"]),
                               down=pack(s["down"]),
                               shared_gate_up=pack(s["shared_gate_up"]) if shared else None,
                               shared_down=pack(s["shared_down"]) if shared else None)
    h.update(desc=desc.c(), w=h["weights"].c(), groups=None,
             workspace=new(B.moe_quant_workspace_size(desc), dtype=torch.uint8))
    if layer:
        h["out"] = new(c["T"], c["H"], dtype=BF16)
        if c["groups"]:
            h["groups"] = B.GroupRoute(n_groups=c["groups"], groups_kept=c["kept"],
                                       group_best=c["best"], select_bias=s["bias"]).c()
    else:
        h["y"] = new(c["T"] * c["k"], c["H"], dtype=BF16)
    return h


def _own_project(state):
    h = state["handle"]
    B = h["B"]
    B.check(B.moe_quant_project(h["desc"], state["x"], h["w"], h["y"], h["status"], h["workspace"]))
    return h["y"]


def _own_layer(state):
    h = state["handle"]
    B = h["B"]
    B.check(B.moe_layer_forward_quant(h["desc"], h["groups"], h["w"], state["x"], state["router"],
                                   state["k"], None, h["out"], h["status"], h["workspace"]))
    return h["out"]


def _own_experts(state):
    h = state["handle"]
    B = h["B"]
    B.check(B.moe_grouped_ffn_quant(h["desc"], h["w"], state["x"], state["token"], state["offsets"],
                                 h["y"], h["status"], h["workspace"]))
    return h["y"]


# ---------------------------------------------------------------- what a pass cannot do without

def _weight_bytes(count, rows, K, c):
    return float(count) * rows * (K / 2.0 + (K + c["group"] - 1) // c["group"]) + 4.0 * count


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "project":
        K, N = c["K"], c["N"]
        out = N // 2 if c["swiglu"] else N
        return {"bytes": _weight_bytes(1, N, K, c) + 2.0 * T * (K + out), "flops": 2.0 * T * K * N}
    H, E, I, k = c["H"], c["E"], c["I"], c["k"]  # noqa: E741
    mean = k if c["op"] == "experts" else ((k + 1) // 2 + k) / 2.0
    used = E * (1.0 - (1.0 - mean / E) ** T)          # distinct experts of independent tokens
    b = used * (_weight_bytes(2, I, H, c) + _weight_bytes(1, H, I, c))
    if c["op"] == "experts":
        return {"bytes": b + 2.0 * T * H + 2.0 * T * k * H + 4.0 * T * k,
                "flops": 6.0 * T * k * H * I}
    s = c["shared"]
    if s:
        b += _weight_bytes(2, s, H, c) + _weight_bytes(1, H, s, c)
    return {"bytes": b + 2.0 * E * H + 4.0 * T * H + 4.0 * T,
            "flops": 2.0 * T * H * E + 6.0 * T * mean * H * I + 6.0 * T * H * s}


# ---------------------------------------------------------------- the same in 64 bits

def _matrix64(w, i, c):
    """Matrix i in float64, a code of the even and one of the odd inputs at a time."""
    codes, scales, factor = w
    q, rows = codes[i], codes.shape[1]
    m = torch.zeros(rows, 2 * q.shape[1], dtype=torch.float64, device=DEV)
    for code, v in enumerate(VALUES[c["code"]]):
        m[:, 0::2] += v * (torch.remainder(q, 16) == code)
        m[:, 1::2] += v * (torch.div(q, 16, rounding_mode="floor") == code)
    at = torch.arange(m.shape[1], device=DEV) // c["group"]
    return m * scales[i].double()[:, at] * float(factor[i])


def _ffn64(x, gate, up, down):
    g = x @ gate.t()
    return (g * torch.special.expit(g) * (x @ up.t())) @ down.t()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    x = s["x"].double()
    if c["op"] == "project":
        y = [x @ _matrix64(s["w"], i, c).t() for i in range(2 if c["swiglu"] else 1)]
        return y[0] * torch.special.expit(y[0]) * y[1] if c["swiglu"] else y[0]

    def expert(i, rows):
        return _ffn64(rows, _matrix64(s["gate_up"], 2 * i, c), _matrix64(s["gate_up"], 2 * i + 1, c),
                      _matrix64(s["down"], i, c))

    if c["op"] == "experts":
        at = s["offsets"].tolist()
        return torch.cat([expert(i, x[s["token"][at[i]:at[i + 1]].long()]) for i in range(c["E"])
                          if at[i + 1] > at[i]])
    p, (_, order), _ = _choice64(x @ s["router"].double().t(), s["bias"], c)
    live = torch.arange(c["E"], device=DEV)[None, :] < s["k"][:, None]
    weight = torch.zeros_like(p).scatter_(1, order, torch.gather(p, 1, order) * live)
    if c["renorm"]:
        weight = weight / weight.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for i in range(c["E"]):
        rows = torch.nonzero(weight[:, i] > 0).flatten()
        if rows.numel():
            out[rows] += weight[rows, i:i + 1] * expert(i, x[rows])
    if c["shared"]:
        out += _ffn64(x, _matrix64(s["shared_gate_up"], 0, c), _matrix64(s["shared_gate_up"], 1, c),
                      _matrix64(s["shared_down"], 0, c))
    return out
