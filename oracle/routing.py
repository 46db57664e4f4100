"""Oracle of what stands around the grouped expert layer: the router, the
sort of the tokens by expert, the weighted way back, and their gradients.

TEST INFRASTRUCTURE ONLY.  Only tests/, __graft_entry__.smoke() and the
cpu_baseline leg of bench.py may import this module; the product path never
imports, calls or links it.

Everything is float64 with no intermediate rounding.  Slot s = t * k + j is
token t's j-th choice; an id outside [0, E) routes its slot nowhere.

  route             k largest logits (ties to the lower expert, -inf never),
                    weights p_{e_j} of the row's softmax, or p_{e_j} / sum_i
                    p_{e_i} (renorm)
  route_backward    the weights' gradient at the logits, the choice fixed
  dispatch          off[e] = #{ids < e}, rows[s] = off[id_s] + #{s' < s:
                    id_s' = id_s}, slots the inverse of rows
  combine           Y[t] = base[t] + sum_j w[t][j] Ys[rows[t][j]]
  combine_backward  dYs[rows[t][j]] = w[t][j] dY[t], dw[t][j] = <dY[t],
                    Ys[rows[t][j]]>
"""

from __future__ import annotations

import numpy as np


def route(logits, k: int, renorm: bool):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = [e for e in sorted(range(E), key=lambda e: (-x[t, e], e)) if x[t, e] > -np.inf][:k]
        if not order:
            continue
        p = np.exp(x[t] - x[t, order[0]])
        total = p[order].sum() if renorm else p.sum()
        ids[t, : len(order)] = order
        w[t, : len(order)] = p[order] / total
    return ids, w


def route_backward(logits, ids, dweights, renorm: bool):
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    out = np.zeros((T, E))
    for t in range(T):
        up = np.zeros(E)
        chosen = np.zeros(E, dtype=bool)
        for e, d in zip(ids[t], dweights[t]):
            if 0 <= e < E:
                up[e] += float(d)
                chosen[e] = True
        if not chosen.any():                       # zeros, whatever the logits are
            continue
        inside = chosen if renorm else np.ones(E, dtype=bool)
        top = np.max(x[t][inside], initial=-np.inf)
        if top == -np.inf:
            continue
        p = np.where(inside, np.exp(x[t] - top), 0.0)
        p /= p.sum()
        out[t] = p * (up - (p * up).sum())
    return out


def dispatch(ids, E: int):
    """(off [E + 1], rows [T][k], slots [routed])."""
    ids = np.asarray(ids)
    flat = ids.reshape(-1).astype(np.int64)
    routed = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E:
            routed[e].append(s)
    slots = np.array([s for group in routed for s in group], dtype=np.int32)
    off = np.concatenate([[0], np.cumsum([len(g) for g in routed])]).astype(np.int32)
    rows = np.full(flat.shape, -1, dtype=np.int32)
    rows[slots] = np.arange(slots.size)
    return off, rows.reshape(ids.shape), slots


def combine(Ys, rows, weights=None, base=None):
    Ys = np.asarray(Ys, dtype=np.float64)
    T, k = rows.shape
    Y = np.zeros((T, Ys.shape[1])) if base is None else np.array(base, dtype=np.float64)
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < Ys.shape[0]:
                Y[t] += (1.0 if weights is None else float(weights[t, j])) * Ys[rows[t, j]]
    return Y


def combine_backward(dY, Ys, rows, weights=None):
    """(dYs, with NaN in the rows that no slot names; dweights)."""
    dY, Ys = np.asarray(dY, dtype=np.float64), np.asarray(Ys, dtype=np.float64)
    T, k = rows.shape
    dYs, dw = np.full(Ys.shape, np.nan), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = rows[t, j]
            if 0 <= r < Ys.shape[0]:
                dYs[r] = (1.0 if weights is None else float(weights[t, j])) * dY[t]
                dw[t, j] = dY[t] @ Ys[r]
    return dYs, dw
