"""Float64 oracle of the adapters of many requests (include/salr.h,
salr_adapters_forward and salr_adapters_backward): token by token.

a [count][r][K] and b [count][N][r] as stored, ids [M], ranks and scales
[count]."""

import numpy as np


def _tokens(ids, count):
    return [(t, int(a)) for t, a in enumerate(ids) if 0 <= a < count]


def forward(a, b, ids, ranks, scales, X, base):
    """Y [M][N]."""
    Y = np.array(base, dtype=np.float64)
    for t, q in _tokens(ids, len(a)):
        n = ranks[q]
        Y[t] += scales[q] * (b[q][:, :n] @ (a[q][:n] @ X[t]))
    return Y


def backward(a, b, ids, ranks, scales, X, dY, base):
    """(dX [M][K], dA [count][r][K], dB [count][N][r])."""
    dX = np.array(base, dtype=np.float64)
    dA, dB = np.zeros(a.shape), np.zeros(b.shape)
    for t, q in _tokens(ids, len(a)):
        n = ranks[q]
        T, G = a[q][:n] @ X[t], scales[q] * (dY[t] @ b[q][:, :n])
        dX[t] += G @ a[q][:n]
        dA[q][:n] += np.outer(G, X[t])
        dB[q][:, :n] += scales[q] * np.outer(dY[t], T)
    return dX, dA, dB


def plan(ids, count):
    """(offsets [count + 2], order [M]): the tokens sorted by adapter, those
    without one last, each group in token order."""
    g = np.array([q if 0 <= q < count else count for q in ids], dtype=np.int64)
    order = np.array([t for q in range(count + 1) for t in range(len(g)) if g[t] == q], dtype=np.int64)
    return np.array([(g < q).sum() for q in range(count + 2)], dtype=np.int64), order
