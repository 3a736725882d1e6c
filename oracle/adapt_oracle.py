"""Plain 64-bit projection with a low-rank adapter per token."""
import numpy as np


def adapted(x, w, a, b, scale, ids):
    """x [tokens][hidden], w [n_out][hidden], a [n][rank][hidden], b [n][n_out][rank], all float64:
    y, and for each output the sums of magnitudes of its two products (shared, adapter's)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = x @ w.T
    size, low = np.abs(x) @ np.abs(w).T, np.zeros_like(y)
    for i in sorted(set(int(v) for v in ids)):
        if not 0 <= i < len(a):
            continue
        rows = np.flatnonzero(np.asarray(ids) == i)
        y[rows] += scale[i] * ((x[rows] @ a[i].T) @ b[i].T)
        low[rows] = abs(scale[i]) * ((np.abs(x[rows]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return y, size, low
