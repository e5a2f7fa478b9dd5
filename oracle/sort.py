"""Oracle of the token-sorting operators (plan, permute, unpermute and their
gradients), entry by entry in float64.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``.  Source: "Nemotron Kernels
From Inference To Backpropagation" -- "Kernel 4: Routed ReLU2 MoE" (select, execute,
weight and combine).
"""

from __future__ import annotations

import numpy as np


def rows_bound(T, k, experts, pad):
    n = T * k
    return -(-(n + min(experts, n) * (pad - 1)) // pad) * pad


def plan(idx, experts, pad):
    """count, seg, pos, row_map of expert ids [T, k]."""
    idx = np.asarray(idx)
    T, k = idx.shape
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(idx.reshape(-1)):
        if 0 <= e < experts:
            lists[e].append(i)
    count = np.array([len(x) for x in lists], dtype=np.int32)
    seg = np.zeros(experts + 1, dtype=np.int32)
    pos = np.full(T * k, -1, dtype=np.int32)
    row_map = np.full(rows_bound(T, k, experts, pad), -1, dtype=np.int32)
    for e, entries in enumerate(lists):
        seg[e + 1] = seg[e] + -(-len(entries) // pad) * pad
        for rank, i in enumerate(entries):
            pos[i] = seg[e] + rank
            row_map[seg[e] + rank] = i
    return count, seg, pos.reshape(T, k), row_map


def permute(x, row_map, k):
    out = np.zeros((len(row_map), x.shape[1]))
    for r, i in enumerate(row_map):
        if i >= 0:
            out[r] = x[i // k]
    return out


def permute_backward(d_rows, pos):
    dx = np.zeros((pos.shape[0], d_rows.shape[1]))
    for t in range(pos.shape[0]):
        for p in pos[t]:
            if p >= 0:
                dx[t] += d_rows[p]
    return dx


def unpermute(rows, pos, weights=None, residual=None):
    """y and the sum of the magnitudes that make it."""
    T, k = pos.shape
    y = np.zeros((T, rows.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    mag = np.abs(y)
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                v = (1.0 if weights is None else float(weights[t, j])) * rows[pos[t, j]]
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag


def unpermute_backward(dy, rows, pos, row_map, weights=None):
    """d_rows, d_weights and the sums of |dy||rows| behind d_weights."""
    T, k = pos.shape
    d_rows = np.zeros((len(row_map), dy.shape[1]))
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if p >= 0:
                d_rows[p] = (1.0 if weights is None else float(weights[t, j])) * dy[t]
                dw[t, j] = dy[t] @ rows[p]
                mag[t, j] = np.abs(dy[t]) @ np.abs(rows[p])
    return d_rows, dw, mag
