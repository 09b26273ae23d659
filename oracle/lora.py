"""A shared projection with a low-rank adapter per token, in float64, token
group by token group.  Returns the result and the sums of absolute terms that
its tolerance is made of.  Test infrastructure."""
import numpy as np


def project(x, w, a, b, ranks, scales, adapter, swiglu=False):
    """(y, base magnitude, adapter magnitude), the magnitudes of the value
    before the SwiGLU."""
    y = x @ w.T
    base = np.abs(x) @ np.abs(w).T
    low = np.zeros_like(y)
    for i in range(len(ranks)):
        rows = np.nonzero(adapter == i)[0]
        r = int(ranks[i])
        if len(rows) and r > 0:
            v = float(scales[i]) * (x[rows] @ a[i, :r].T)
            y[rows] += v @ b[i][:, :r].T
            low[rows] = np.abs(v) @ np.abs(b[i][:, :r]).T
            base[rows] += abs(float(scales[i])) * (np.abs(x[rows]) @ np.abs(a[i, :r]).T) @ np.abs(
                b[i][:, :r]).T
    if not swiglu:
        return y, base, low
    return swiglu_of(y), base, low


def swiglu_of(y):
    n = y.shape[1] // 2
    g, u = y[:, :n], y[:, n:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
