"""Group-limited routing with a balance bias, in float64, token by token.

Written from the formulas: score, biased score, group rank (sum of the
`best` largest biased scores), the kept groups, the k_t best units inside
them, their weights; and the gradient of the weights.  Test infrastructure.
"""
import math

import numpy as np


def scores(logits, score):
    """float64 scores; units out of service (not below +inf, or -inf) score 0."""
    l = np.asarray(logits, dtype=np.float64)
    live = l < np.inf
    l = np.where(live, l, -np.inf)
    live = l > -np.inf
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0), live
    if not live.any():
        return np.zeros_like(l), live
    e = np.where(live, np.exp(np.where(live, l, 0.0) - l[live].max()), 0.0)
    return e / e.sum(), live


def route_token(logits, k, score, renorm, scale, n_groups=1, kept=1, best=1, bias=None):
    """(units, weights, gap) of one token; gap: the least difference of two
    values that a decision compared."""
    s, live = scores(logits, score)
    E = len(s)
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    c = np.where(live & (b > -np.inf), s + b, -np.inf)
    size = E // n_groups
    gap = math.inf
    rank = []
    for g in range(n_groups):
        top = sorted((v for v in c[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:best]
        rank.append(sum(top) if top else -math.inf)
    order = sorted(range(n_groups), key=lambda g: (-rank[g], g))
    if kept < n_groups and rank[order[kept]] > -math.inf:
        if rank[order[kept - 1]] != rank[order[kept]]:
            gap = min(gap, rank[order[kept - 1]] - rank[order[kept]])
    inside = [u for g in order[:kept] for u in range(g * size, (g + 1) * size) if c[u] > -np.inf]
    inside.sort(key=lambda u: (-c[u], u))
    chosen = inside[:k]
    for a, d in zip(inside[:k], inside[1:k + 1]):
        if c[a] != c[d]:
            gap = min(gap, c[a] - c[d])
    w = s[chosen]
    if renorm and len(chosen):
        if score == "softmax":     # the softmax of the selected logits
            l = np.asarray(logits, dtype=np.float64)[chosen]
            e = np.exp(l - l.max())
            w = e / e.sum()
        else:
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
    return chosen, scale * w, gap


def route_backward_token(logits, idx, d_w, score, renorm, scale):
    """Gradient at the logits, and the sum of the absolute terms it is made of."""
    s, live = scores(logits, score)
    E = len(s)
    d, mag = np.zeros(E), np.zeros(E)
    use = [(j, u) for j, u in enumerate(idx) if u >= 0 and live[u]]
    if not use:
        return d, mag
    js, us = [j for j, _ in use], [u for _, u in use]
    g = scale * np.asarray(d_w, dtype=np.float64)[js]
    if not renorm:
        ds = np.zeros(E)
        ds[us] = g
        if score == "sigmoid":
            return s * (1 - s) * ds, s * np.abs(ds)
        return s * (ds - (ds * s).sum()), s * (np.abs(ds) + (np.abs(ds) * s).sum())
    l = np.asarray(logits, dtype=np.float64)[us]
    if score == "softmax":
        e = np.exp(l - l.max())
        w, factor = e / e.sum(), np.ones(len(us))
    else:
        w = s[us] / s[us].sum() if s[us].sum() > 0 else np.zeros(len(us))
        factor = 1 - s[us]
    d[us] = w * factor * (g - (g * w).sum())
    mag[us] = w * factor * (np.abs(g) + (np.abs(g) * w).sum())
    return d, mag
