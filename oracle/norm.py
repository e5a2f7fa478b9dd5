"""Float64 oracle of the residual sum with RMSNorm and E4M3 codes ("Nemotron Kernels From
Inference To Backpropagation" -- "Setup: The Shared Transformer Shell", "Where
Quantization Fits"; "Reverse-mode automatic differentiation" section 5)."""

from __future__ import annotations

import numpy as np

MAX = 448.0


def _blocks(width, block):
    return [(c, min(c + block, width)) for c in range(0, width, block)] if block else [(0, width)]


def e4m3(v):
    """The nearest E4M3 value, ties to even, saturated."""
    a = np.abs(v)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, MAX), v)


def forward(s, gamma, eps, block=0):
    """n, the codes' values [T, width] (before the scale), scales [T, blocks] as float32, rstd of the kept sum s."""
    s, gamma = np.asarray(s, dtype=np.float64), np.asarray(gamma, dtype=np.float64)
    r = 1.0 / np.sqrt((s * s).mean(axis=1) + np.float64(np.float32(eps)))
    n = s * r[:, None] * gamma
    codes, scales = np.zeros_like(n), []
    for c, d in _blocks(s.shape[1], block):
        top = np.abs(n[:, c:d]).max(axis=1)
        scale = np.where(top > 0, top / MAX, 1.0).astype(np.float32)
        scales.append(scale)
        codes[:, c:d] = e4m3(n[:, c:d] / scale.astype(np.float64)[:, None])
    return n, codes, np.stack(scales, axis=1), r


def backward(dn, s, gamma, r, d_sum=None):
    """dx and dgamma."""
    dn, s, gamma = (np.asarray(v, dtype=np.float64) for v in (dn, s, gamma))
    xh = s * r[:, None]
    g = dn * gamma
    dx = r[:, None] * (g - xh * (g * xh).mean(axis=1, keepdims=True))
    return (dx if d_sum is None else dx + d_sum), (dn * xh).sum(axis=0)
