"""Float64 oracle of the orthogonalised update: Newton-Schulz steps on a matrix, and Muon's
step (K. Jordan et al., 2024; "optimizer state": one moment per weight)."""

from __future__ import annotations

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, coefficients=(COEFFICIENTS,) * 5, eps=1e-7):
    """One matrix."""
    x = np.asarray(u, dtype=np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    for a, b, c in coefficients:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def muon_step(w, m, g, lr, beta, wd=0.0, scale=1.0, nesterov=True, **kw):
    """New weight and momentum of one matrix."""
    m = beta * m + g
    x = orthogonalize(g + beta * m if nesterov else m, **kw)
    return w * (1.0 - lr * wd) - lr * scale * x, m
