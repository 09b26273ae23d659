"""4-bit weights with group scales, and products with them, in float64.  Returns
results and what their tolerances are made of.  Test infrastructure."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
INT4 = np.arange(16.0) - 8.0
VALUES = {"e2m1": E2M1, "int4": INT4}

STEP = 2.0 ** -8          # bf16: half a step, relative


def e4m3(bits):
    """Values of e4m3 bytes (NaN for the one pattern that is)."""
    b = np.asarray(bits, dtype=np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6.0)
    return np.where((b & 127) == 127, np.nan, np.where(b & 128, -v, v))


def weights(codes, scales, factors, kind, group):
    """codes uint8 [count, rows, K / 2], scales e4m3 bytes, factors -> [count, rows, K]."""
    q = np.stack((codes & 15, codes >> 4), axis=-1).reshape(codes.shape[0], codes.shape[1], -1)
    s = np.repeat(e4m3(scales), group, axis=2)[..., :q.shape[-1]]
    return VALUES[kind][q] * s * np.asarray(factors, dtype=np.float64)[:, None, None]


def product(x, w, dx=0.0):
    """x w^T and a bound of its error in fp32 sums, x off by at most dx.  A sum of n terms in
    any order, each addition within 2^-23 of its value (tensor cores cut off, they do not round)."""
    mag = np.abs(x) @ np.abs(w).T
    return x @ w.T, (w.shape[1] + 4) * 2.0 ** -23 * mag + np.broadcast_to(dx, x.shape) @ np.abs(w).T


def swiglu(g, dg, u, du):
    """silu(g) u and its error: silu has a slope of at most 1.1; the fp32 sigmoid's own error is
    within (4 + 1.2 |g|) 2^-23 of its value."""
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    y = s * u
    return y, 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + (6 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(y)


def rounded(y, dy):
    """A value that is off by dy, rounded to bf16."""
    return dy + STEP * (np.abs(y) + dy)


def ffn(x, gate, up, down):
    """SwiGLU FFN, its activations rounded to bf16: (y, bound before y's own rounding)."""
    a, da = swiglu(*product(x, gate), *product(x, up))
    return product(a, down, rounded(a, da))
