"""The router against the oracle (oracle.route), GB300 only.

ids are compared exactly: the order is that of the scores in float64.  Weights: a score is
off by at most exp's ulp (2^-23), the rounding of its argument l - m (|l - m| * 2^-24 of the
value), the sum of its E terms (E + 1 roundings) and a quotient; a renormalised weight by the
same once more and the sum of its k terms: all in half steps of 2^-24.  Gradients: the same
on the magnitudes that they are made of, and half a step of their type (bf16 2^-8).
"""

import numpy as np
import pytest

from oracle import route
from helpers import to_dev, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mb():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mlp_block_backprop_gb300 as mb
    yield mb
    assert mb.mlpblk_last_error() == mb.MLPBLK_OK


def _logits(rng, T, E, kind, dtype):
    """As the kernel gets them: float32 values of the dtype."""
    import torch
    l = rng.normal(0, 1.5, (T, E))
    if kind == "ties":
        l = np.round(l)                                   # many equal logits
    elif kind == "masked":
        l[rng.random((T, E)) < 0.4] = -np.inf
        l[rng.random(T) < 0.3] = -np.inf                  # rows that nothing is left of
        l[rng.random((T, E)) < 0.02] = np.nan
        l[rng.random((T, E)) < 0.02] = np.finfo(np.float32).min
    elif kind == "far":
        l = rng.normal(0, 60, (T, E))                     # most scores vanish
        l[rng.random((T, E)) < 0.02] = np.inf
    elif kind == "near":
        l = 0.5 + rng.integers(0, 3, (T, E)) * 2.0 ** -24 + rng.integers(0, 2, (T, E))   # neighbours in float32
    t = torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.cuda(), t.float().numpy()


def _tol(logits, E, k):
    """Relative bound of a weight."""
    l = np.where(np.isfinite(logits), logits, 0.0)
    far = np.minimum(np.abs(l.max(axis=1) - l.min(axis=1)), 110.0).max()   # beyond, exp is zero in float32
    return (2 * (far + 2 + E + 2) + k + 3) * U


CASES = [
    # T, E, k, score, groups, top_groups, renorm, scale
    (1, 1, 1, "softmax", 1, 1, True, 1.0),
    (5, 8, 8, "softmax", 1, 1, False, 1.0),
    (7, 3, 2, "sigmoid", 1, 1, True, 2.5),
    (130, 8, 2, "softmax", 1, 1, True, 1.0),
    (33, 12, 3, "softmax", 4, 2, True, 1.0),
    (65, 16, 4, "sigmoid", 2, 1, False, 0.5),
    (257, 30, 5, "sigmoid", 5, 3, True, 1.0),
    (100, 60, 6, "softmax", 1, 1, True, 1.0),
    (64, 64, 8, "sigmoid", 8, 4, True, 2.0),
    (31, 100, 16, "softmax", 4, 4, False, 1.0),
    (50, 128, 8, "softmax", 64, 7, True, 1.0),
    (40, 255, 16, "softmax", 1, 1, True, 1.0),
    (300, 256, 8, "sigmoid", 8, 4, True, 2.5),
    (77, 256, 1, "softmax", 1, 1, True, 1.0),
    (20, 250, 7, "sigmoid", 10, 3, False, 1.0),
]


@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "far", "near"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_route_and_gradient(mb, case, dtype, biased, kind):
    import torch
    T, E, k, score, groups, top_groups, renorm, scale = case
    rng = np.random.default_rng(T * E + k)
    dev, l = _logits(rng, T, E, kind, dtype)
    bias = (np.round(rng.normal(0, 0.1, E), 1) if kind == "ties" else rng.normal(0, 0.1, E)).astype(np.float32) if biased else None
    r = mb.MoeRouter(T, E, k, score, groups, top_groups, renorm, scale, dtype)
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 77.0, device="cuda")
    r.route(dev, ids, w, bias=None if bias is None else torch.from_numpy(bias).cuda())
    ref_ids, ref_w = route.route(l, k, score, bias, groups, top_groups, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    tol = _tol(l, E, k)
    got = to_np(w)
    # (float32 scores below its normal range lose their last bits, and a sum of such is compared with 1e-20)
    assert np.all(np.abs(got - ref_w) <= tol * np.abs(ref_w) + 2.0 ** -126 * (1 if not renorm else 1e20)), np.abs(got - ref_w).max()

    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    dl = torch.full((T, E), float("nan"), dtype=dev.dtype, device="cuda")
    r.route_backward(dev, ids, torch.from_numpy(dw).cuda(), dl)
    ref = route.backward(l, ref_ids, dw, score, renorm, scale)
    # the magnitudes of what is added: |ds| s and, of a dense softmax, s sum |ds| s
    mag = np.zeros((T, E))
    for t in range(T):
        s = route.scores(l[t], score)
        e = [i for i in ref_ids[t] if i >= 0]
        g = np.abs(scale * dw[t, :len(e)].astype(np.float64))
        if renorm:
            S = s[e].sum() + route.TINY
            g = (g + (g * s[e]).sum() / S) / S
        mag[t, e] = g * s[e]
        if score == "softmax" and not renorm:
            mag[t] += s * (g * s[e]).sum()
    half = 2.0 ** -8 if dtype == "bf16" else U
    floor = 2.0 ** -126 * (1 if not renorm else 1e20) * max(1.0, np.abs(scale * dw).max())
    err = np.abs(to_np(dl) - ref)
    assert np.all(err <= 4 * tol * mag + half * np.abs(ref) + floor), (err - 4 * tol * mag - half * np.abs(ref)).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", [c for c in CASES if c[1] > 1])
def test_biases_that_are_not_finite(mb, case, dtype):
    """-inf and NaN close an expert to selection, +inf puts it first; more of each than are selected.
    The others' biases are zero, so that many keys are equal, and equal in float32 alone."""
    import torch
    T, E, k, score, groups, top_groups, renorm, scale = case
    rng = np.random.default_rng(T + E)
    for kind in ("plain", "ties", "near", "far"):
        dev, l = _logits(rng, T, E, kind, dtype)
        for values in ((), (np.inf,), (-np.inf, np.nan), (np.inf, -np.inf, np.nan)):
            bias = np.zeros(E, dtype=np.float32)
            for i, v in enumerate(values):
                bias[rng.random(E) < (0.15 if np.isposinf(v) and kind == "plain" else 0.5)] = v
            ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
            w = torch.full((T, k), 77.0, device="cuda")
            mb.MoeRouter(T, E, k, score, groups, top_groups, renorm, scale, dtype).route(dev, ids, w, bias=torch.from_numpy(bias).cuda())
            ref_ids, ref_w = route.route(l, k, score, bias, groups, top_groups, renorm, scale)
            np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
            np.testing.assert_allclose(to_np(w), ref_w, rtol=_tol(l, E, k), atol=2.0 ** -126 * (1 if not renorm else 1e20))


def test_gradient_against_differences(mb):
    """d_logits on central differences of L = sum dw w in float32 steps that keep the selection."""
    import torch
    T, E, k = 6, 24, 4
    rng = np.random.default_rng(3)
    l = torch.from_numpy(rng.normal(0, 1, (T, E)).astype(np.float32)).cuda()
    dw = torch.from_numpy(rng.normal(0, 1, (T, k)).astype(np.float32)).cuda()
    for score, renorm in (("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)):
        r = mb.MoeRouter(T, E, k, score, renorm=renorm, scale=1.5, dtype="f32")
        ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
        r.route(l, ids, w)
        dl = torch.empty_like(l)
        r.route_backward(l, ids, dw, dl)
        h = 2.0 ** -7
        for t in range(T):
            for e in list(ids[t].cpu().numpy()) + [int(e) for e in range(E) if e not in ids[t].tolist()][:3]:
                side = []
                for sign in (1, -1):
                    x = l.clone()
                    x[t, e] += sign * h
                    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
                    r.route(x, i2, w2)
                    if sorted(i2[t].tolist()) != sorted(ids[t].tolist()):
                        break
                    by = {int(a): float(b) for a, b in zip(i2[t], w2[t])}
                    side.append(sum(float(dw[t, j]) * by[int(ids[t, j])] for j in range(k)))
                if len(side) == 2:
                    # third derivatives are below 1.5 |dw| k; a weight is off by 2^-20
                    bound = 6 * h * h * k + 2 * 3 * k * 2.0 ** -20 / h
                    assert abs((side[0] - side[1]) / (2 * h) - float(dl[t, e])) <= bound


def test_repeats_are_bitwise_equal(mb):
    import torch
    rng = np.random.default_rng(5)
    dev, _ = _logits(rng, 3000, 256, "near", "f32")
    bias = torch.from_numpy(rng.normal(0, 0.1, 256).astype(np.float32)).cuda()
    r = mb.MoeRouter(3000, 256, 8, "sigmoid", 8, 4, dtype="f32")
    out = []
    for _ in range(3):
        ids, w, dl = torch.empty(3000, 8, dtype=torch.int32, device="cuda"), torch.empty(3000, 8, device="cuda"), torch.empty_like(dev)
        r.route(dev, ids, w, bias=bias)
        r.route_backward(dev, ids, torch.ones_like(w).cumsum(1), dl)
        out.append((ids, w, dl))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], o))


def test_ids_of_another_router_stay_inside(mb):
    """Ids outside the experts have no gradient and are not used as addresses."""
    import torch
    T, E, k = 50, 20, 4
    r = mb.MoeRouter(T, E, k, "softmax", dtype="bf16")
    rng = np.random.default_rng(7)
    dev, l = _logits(rng, T, E, "plain", "bf16")
    ids = rng.choice([-1, -7, E, 1 << 30, 3, 5], (T, k)).astype(np.int32)
    for t in range(T):   # no expert twice
        for j in range(k):
            if ids[t, j] in (3, 5) and ids[t, j] in ids[t, :j]:
                ids[t, j] = -1
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    dl = torch.full((T, E), float("nan"), dtype=torch.bfloat16, device="cuda")
    r.route_backward(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), dl)
    ref = route.backward(l, ids, dw, "softmax")
    np.testing.assert_allclose(to_np(dl), ref, rtol=2.0 ** -7, atol=1e-5)


def test_capture_on_another_stream_and_replay(mb):
    import torch
    T, E, k = 500, 64, 6
    rng = np.random.default_rng(11)
    dev, _ = _logits(rng, T, E, "plain", "bf16")
    r = mb.MoeRouter(T, E, k, "sigmoid", dtype="bf16")
    ids, w, dl = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty_like(dev)
    r.route(dev, ids, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.route(dev, ids, w)
        r.route_backward(dev, ids, w, dl)
    new, l = _logits(rng, T, E, "ties", "bf16")
    dev.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    ref_ids, ref_w = route.route(l, k, "sigmoid")
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    np.testing.assert_allclose(to_np(w), ref_w, rtol=_tol(l, E, k))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_offsets_beyond_32_bits(mb, score):
    """2^32 logits and more: the last tokens as a batch of their own."""
    import torch
    E, k = 256, 4
    T, last = (1 << 24) + 77, 100
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    bias = torch.randn(E, device="cuda") * 0.1
    ids, w = torch.full((T, k), 77, dtype=torch.int32, device="cuda"), torch.full((T, k), 77.0, device="cuda")
    mb.MoeRouter(T, E, k, score).route(l, ids, w, bias=bias)
    dw, dl = torch.randn(T, k, device="cuda"), torch.full((T, E), 77.0, dtype=torch.bfloat16, device="cuda")
    mb.MoeRouter(T, E, k, score, renorm=False).route_backward(l, ids, dw, dl)
    n = T - last
    tail = l[n:].clone()
    ids2, w2, dl2 = torch.empty_like(ids[n:]), torch.empty_like(w[n:]), torch.empty_like(tail)
    mb.MoeRouter(last, E, k, score).route(tail, ids2, w2, bias=bias)
    mb.MoeRouter(last, E, k, score, renorm=False).route_backward(tail, ids2, dw[n:].clone(), dl2)
    assert torch.equal(ids[n:], ids2) and torch.equal(w[n:], w2) and torch.equal(dl[n:], dl2)
    ref_ids, _ = route.route(to_np(tail), k, score, to_np(bias))
    np.testing.assert_array_equal(ids2.cpu().numpy(), ref_ids)
