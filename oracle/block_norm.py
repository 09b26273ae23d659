"""The norms around a residual block and their gradients, in float64.

r' = rs r + bs g z, z = w_post' y / rms(y), h = w_pre' r' / rms(r').  The
backward pass also returns, per output, a bound on the size of the terms it
sums, for tolerances.  Test infrastructure.
"""
import numpy as np


def _rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate(gate, kind, shape):
    if kind == "none":
        return np.ones(shape)
    if kind == "token":
        return np.broadcast_to(gate[:, None], shape)
    return np.broadcast_to(gate, shape)


def forward(r, y=None, gate=None, kind="none", w_post=None, w_pre=None, offset=0.0, rs=1.0, bs=1.0,
            eps=1e-6):
    """(r', h or None, magnitude of r')."""
    if y is None:
        out, mag = rs * r, np.abs(rs * r)
    else:
        z = y if w_post is None else y * _rstd(y, eps) * (w_post + offset)
        b = bs * _gate(gate, kind, r.shape) * z
        out, mag = rs * r + b, np.abs(rs * r) + np.abs(b)
    if w_pre is None:
        return out, None, mag
    return out, out * _rstd(out, eps) * (w_pre + offset), mag


def backward(r, y, gate, kind, w_post, w_pre, d_out, d_h, offset=0.0, rs=1.0, bs=1.0, eps=1e-6):
    """{name: (gradient, size of its terms)}."""
    got = {}
    out = forward(r, y, gate, kind, w_post, None, offset, rs, bs, eps)[0]
    D = np.zeros_like(r) if d_out is None else d_out.copy()
    size = np.abs(D)
    if w_pre is not None:
        f = _rstd(out, eps)
        m, dm = out * f, d_h * (w_pre + offset)
        D = D + f * (dm - m * (dm * m).mean(axis=1, keepdims=True))
        size = size + f * (np.abs(dm) + np.abs(m) * np.abs(dm * m).mean(axis=1, keepdims=True))
        got["d_w_pre"] = ((d_h * m).sum(0), np.abs(d_h * m).sum(0))
    got["d_residual"] = (rs * D, abs(rs) * size)
    if y is None:
        return got
    g = _gate(gate, kind, r.shape)
    f = _rstd(y, eps) if w_post is not None else 1.0
    n = y * f
    z = n if w_post is None else n * (w_post + offset)
    dz, zs = bs * D * g, abs(bs) * size * np.abs(g)
    dg, gs = bs * D * z, abs(bs) * size * np.abs(z)
    if kind == "channel":
        got["d_gate"] = (dg.sum(0), gs.sum(0))
    elif kind == "token":
        got["d_gate"] = (dg.sum(1), gs.sum(1))
    elif kind == "full":
        got["d_gate"] = (dg, gs)
    if w_post is None:
        got["d_branch"] = (dz, zs)
        return got
    got["d_w_post"] = ((dz * n).sum(0), (zs * np.abs(n)).sum(0))
    dn, ns = dz * (w_post + offset), zs * np.abs(w_post + offset)
    got["d_branch"] = (f * (dn - n * (dn * n).mean(axis=1, keepdims=True)),
                       f * (ns + np.abs(n) * (ns * np.abs(n)).mean(axis=1, keepdims=True)))
    return got
