"""Float64 oracle of the router: logits -> expert ids and weights, and the logits'
gradient ("Nemotron Kernels From Inference To Backpropagation" -- "Kernel 4: Routed ReLU2
MoE": select), token by token in the order of the definition."""

from __future__ import annotations

import numpy as np

TINY = 1e-20


def _row(logits):
    """A row as the formulas take it: NaN and -inf closed, +inf the largest float32."""
    l = np.asarray(logits, dtype=np.float64)
    return np.where(l > -np.inf, np.minimum(l, np.finfo(np.float32).max), -np.inf)


def scores(logits, score):
    l = _row(logits)
    live = l > -np.inf
    s = np.zeros_like(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    elif live.any():
        e = np.exp(l[live] - l[live].max())
        s[live] = e / e.sum()
    return s


def _order(values):
    """Indices by descending value, ties to the lower index, without the -inf ones."""
    return [i for i in sorted(range(len(values)), key=lambda i: (-values[i], i)) if values[i] > -np.inf]


def route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, renorm=True, scale=1.0):
    """ids [T, k] int32 and weights [T, k]."""
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    ids, weights = np.full((T, top_k), -1, dtype=np.int32), np.zeros((T, top_k))
    for t in range(T):
        s, l = scores(logits[t], score), _row(logits[t])
        b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
        key = np.where((l > -np.inf) & (b > -np.inf), s + b, -np.inf)
        rank = l if bias is None else key          # without a bias the logits decide
        if top_groups < groups:
            per = E // groups
            marks = []
            for g in range(groups):
                best = [key[e] for e in range(g * per, (g + 1) * per) if key[e] > -np.inf]
                marks.append(sum(sorted(best)[-2:]) if best else -np.inf)
            keep = sorted(range(groups), key=lambda g: (-marks[g], g))[:top_groups]
            rank = np.array([rank[e] if e // per in keep else -np.inf for e in range(E)])
        chosen = _order(rank)[:top_k]
        ids[t, :len(chosen)] = chosen
        w = s[chosen]
        weights[t, :len(chosen)] = scale * (w / (w.sum() + TINY) if renorm else w)
    return ids, weights


def backward(logits, ids, d_weights, score="softmax", renorm=True, scale=1.0):
    """d_logits, the ids held fixed."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        s, l = scores(logits[t], score), _row(logits[t])
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and l[ids[t, j]] > -np.inf]
        e = [ids[t, j] for j in slots]
        g = scale * np.asarray(d_weights, dtype=np.float64)[t, slots]
        mean = (g * s[e]).sum()                     # sum_j ds_j s_j
        if renorm:
            S = s[e].sum() + TINY
            g = (g - mean / S) / S
            mean = mean / S * (TINY / S)            # the same sum: of S - TINY against S
        ds = np.zeros(E)
        np.add.at(ds, e, g)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                out[t] = ds * s * np.where(l > -np.inf, 1.0 / (1.0 + np.exp(l)), 0.0)
        else:
            out[t] = s * (ds - mean)
    return out
