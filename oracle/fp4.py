"""Float64 oracle of the MXFP4 format (OCP Microscaling Formats specification:
blocks of 32 E2M1 elements with a shared E8M0 scale), its byte layout in this
library and the products of quantised matrices.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``: the CUDA library never
calls it and shares no code with it.

Readings: the shared exponent is floor(log2(max |v|)) - 2 (the specification's
rule; 2 is the exponent of E2M1's largest binade), at least -127; elements round to
nearest even and saturate at 6; a block with an infinity or NaN reads back as NaN.
"""

from __future__ import annotations

import numpy as np

VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def e2m1(u):
    """Code (0..15) of each value: the nearest of VALUES, the even code on a tie."""
    u = np.asarray(u, dtype=np.float64)
    d = np.abs(np.abs(u)[..., None] - VALUES)
    best = d.min(axis=-1, keepdims=True)
    near = d == best                               # one candidate, or two on a tie
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (code + 8 * np.signbit(u)).astype(np.uint8)


def decode(code):
    code = np.asarray(code)
    return np.where(code >= 8, -1.0, 1.0) * VALUES[code % 8]


def quantize(v):
    """(codes [rows, 32 * blocks], scale bytes [rows, blocks]) of a matrix."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    nb = -(-cols // BLOCK)
    w = np.zeros((rows, nb * BLOCK))
    w[:, :cols] = v
    w = w.reshape(rows, nb, BLOCK)
    top = np.abs(w).max(axis=2)
    bad = ~np.isfinite(w).all(axis=2)
    e = np.full(top.shape, -127.0)
    pos = np.isfinite(top) & (top > 0)
    e[pos] = np.maximum(np.frexp(top[pos])[1] - 1 - 2, -127)
    codes = e2m1(np.where(bad[..., None], 0.0, np.ldexp(np.where(bad[..., None], 0.0, w), -e.astype(int)[..., None])))
    sb = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(rows, nb * BLOCK), sb


def values(codes, scales, cols):
    """The matrix that codes and scale bytes stand for."""
    rows, nb = scales.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (decode(codes).reshape(rows, nb, BLOCK) * s[..., None]).reshape(rows, -1)[:, :cols]


def rounded(v):
    c, s = quantize(v)
    return values(c, s, np.asarray(v).shape[1])


def pack(codes, scales):
    """The two byte buffers of the library's layout."""
    rows, nb = scales.shape
    c = codes.reshape(rows, -1, 2)
    packed = (c[..., 0] | (c[..., 1] << 4)).astype(np.uint8).reshape(-1)
    tiles_r, tiles_c = -(-rows // 128), 2 * -(-nb // 8)
    out = np.zeros(tiles_r * tiles_c * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * tiles_c + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = scales
    return packed, out


def product(a, b):
    """A . B^T of two quantised matrices' values, and the sums of |a||b|."""
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    return a @ b.T, np.abs(a) @ np.abs(b).T
