"""The residual norm's gradient and outputs at the ends of float32's range, and with a gamma that is not
finite, against the oracle (oracle.norm), GB300 only.

Tolerances as in test_gpu_norm.py: n three roundings of 2^-24 and half a step of its type; dx half a step,
eight roundings of each summand and width + 3 of the dot product's terms; dgamma tokens + 4.
"""

import numpy as np
import pytest

from oracle import norm
from helpers import to_np

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


def _t(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda().to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [40, 1001, 1024, 4096, 16384])
def test_gradients_of_large_and_small_rows(mb, width, dtype, eps):
    """rstd from 1e-17 to 1e18: its cube leaves float32's range, the gradient does not."""
    import torch
    size = [1e12, 1e14, 1e15, 1e16, 1e17, 1.0] + ([1e-3] if eps else [1e-10, 1e-13, 1e-15, 1e-18])
    T = len(size)
    rng = np.random.default_rng(width)
    # (magnitudes of at most 1.7 times the row's size: the sum of their squares stays in range)
    s = _t(rng.uniform(-1.7, 1.7, (T, width)) * np.array(size)[:, None], dtype)
    dn, gamma = _t(rng.normal(0, 1, (T, width)), dtype), _t(1 + rng.normal(0, 0.2, width), dtype)
    op = mb.AddRmsNorm(T, width, eps, dtype)
    op.forward(s, gamma, n=torch.empty_like(s))
    S, N, G = to_np(s), to_np(dn), to_np(gamma)
    r = to_np(op.rstd)
    np.testing.assert_allclose(r, 1 / np.sqrt((S * S).mean(axis=1) + np.float64(np.float32(eps))), rtol=2.0 ** -23)
    dx, dg = torch.full_like(s, float("nan")), torch.full((width,), float("nan"), device="cuda")
    op.backward(dn, s, gamma, dx, dg, overwrite=True)
    ref, ref_dg = norm.backward(N, S, G, r)
    R = r[:, None]
    dots = np.abs(N * G * S * R).mean(axis=1, keepdims=True)
    half = 2.0 ** -8 if dtype == "bf16" else U
    tol = half * np.abs(ref) + 8 * U * (np.abs(N * G) * R + np.abs(S) * R * R * dots) + (width + 3) * U * np.abs(S) * R * R * dots
    err = np.abs(to_np(dx) - ref)
    assert np.all(err <= tol), [(m, float((e / t).max())) for m, e, t in zip(size, err, tol)]
    assert np.all(np.abs(to_np(dg) - ref_dg) <= (T + 4) * U * np.abs(N * S * R).sum(axis=0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
def test_mean_squares_below_the_normal_range(mb, dtype, block):
    """eps = 0 and rows of 2^-65: their squares are 2^-130, exact, and rstd is 2^65."""
    import torch
    T, d = 5, 300
    rng = np.random.default_rng(3)
    x = rng.choice([-1.0, 1.0, 2.0], (T, d)) * 2.0 ** -np.arange(60, 70, 2)[:, None]
    x, gamma = _t(x, dtype), _t(rng.choice([0.5, 1.0, 1.5], d), dtype)
    op = mb.AddRmsNorm(T, d, 0.0, dtype, block)
    codes, n = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty_like(x)
    scales = torch.empty(T, 3 if block else 1, device="cuda")
    op.forward(x, gamma, codes, scales, n=n)
    ref_n, ref_codes, ref_scales, ref_r = norm.forward(to_np(x), to_np(gamma), 0.0, block)
    np.testing.assert_allclose(to_np(op.rstd), ref_r, rtol=2.0 ** -23)
    np.testing.assert_allclose(to_np(n), ref_n, rtol=3 * U + (2.0 ** -8 if dtype == "bf16" else U))
    np.testing.assert_array_equal(to_np(scales), ref_scales.astype(np.float64))
    np.testing.assert_array_equal(to_np(codes), ref_codes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_res", [True, False])
@pytest.mark.parametrize("width", [300, 1024, 5000])
def test_n_where_the_products_of_sum_and_gamma_overflow(mb, width, with_res, dtype):
    """sum * gamma is 2^130, n = sum * rstd * gamma is not: n is the formula's."""
    import torch
    T = 400
    rng = np.random.default_rng(6)
    x, gamma = rng.normal(0, 1, (T, width)), 1 + rng.normal(0, 0.2, width)
    x[3, 200], x[-1, 200], gamma[200] = 2.0 ** 20, -2.0 ** 22, 2.0 ** 110
    res = rng.normal(0, 1, (T, width)) if with_res else None
    x, gamma = _t(x, dtype), _t(gamma, dtype)
    s = torch.empty_like(x) if with_res else None
    op, n = mb.AddRmsNorm(T, width, 1e-6, dtype), torch.empty_like(x)
    op.forward(x, gamma, n=n, residual=_t(res, dtype) if with_res else None, sum=s)
    ref, _, _, _ = norm.forward(to_np(s if with_res else x), to_np(gamma), 1e-6)
    np.testing.assert_allclose(to_np(n), ref, rtol=3 * U + (2.0 ** -8 if dtype == "bf16" else U), atol=1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_gamma_that_is_not_finite(mb, dtype, block, value):
    """max |n| over a NaN or an infinity: the scale of its block (or row) and that scale's codes are NaN, the others are not."""
    import torch
    for T, d, at in ((5, 300, 200), (700, 1024, 1023), (3, 129, 0), (40, 1001, 640)):
        rng = np.random.default_rng(d)
        x, gamma = _t(rng.normal(0, 1, (T, d)), dtype), _t(1 + rng.normal(0, 0.2, d), dtype)
        gamma[at] = value
        per = (d + 127) // 128 if block else 1
        op = mb.AddRmsNorm(T, d, 1e-6, dtype, block)
        codes, scales = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, per, device="cuda")
        op.forward(x, gamma, codes, scales)
        fine = to_np(gamma)
        fine[at] = 1.0
        _, ref_codes, ref_scales, ref_r = norm.forward(to_np(x), fine, 1e-6, block)
        np.testing.assert_allclose(to_np(op.rstd), ref_r, rtol=2.0 ** -23)
        bad = np.zeros(per, dtype=bool)
        bad[at // 128 if block else 0] = True
        wide = np.repeat(bad, 128 if block else d)[:d]
        assert np.isnan(to_np(scales)[:, bad]).all() and np.isnan(to_np(codes)[:, wide]).all()
        np.testing.assert_array_equal(to_np(scales)[:, ~bad], ref_scales.astype(np.float64)[:, ~bad])
        np.testing.assert_array_equal(to_np(codes)[:, ~wide], ref_codes[:, ~wide])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [200, 1536, 5120])
def test_blocks_of_zeros_among_others(mb, width, dtype):
    """Blocks of zeros (also negative ones) and of values below 2^-60 beside ordinary ones, and widths whose last units lie
    behind the row's end: scales of 1 and codes of zero with the values' signs."""
    import torch
    T = 700
    rng = np.random.default_rng(width)
    x = rng.normal(0, 1, (T, width))
    for t in range(T):
        b = rng.integers(0, (width + 127) // 128)
        x[t, 128 * b:128 * (b + 1)] = (0.0, -0.0, 1e-25, 2.0 ** -100)[t % 4]
    x, gamma = _t(x, dtype), _t(1 + rng.normal(0, 0.2, width), dtype)
    op = mb.AddRmsNorm(T, width, 1e-6, dtype, 128)
    codes, scales = torch.empty(T, width, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(T, (width + 127) // 128, device="cuda")
    op.forward(x, gamma, codes, scales)
    _, ref_codes, ref_scales, _ = norm.forward(to_np(x), to_np(gamma), 1e-6, 128)
    np.testing.assert_array_equal(to_np(scales), ref_scales.astype(np.float64))
    np.testing.assert_array_equal(to_np(codes), ref_codes)
    np.testing.assert_array_equal(np.signbit(to_np(codes)), np.signbit(to_np(x)))


@pytest.mark.parametrize("shape", [(52000, 256), (30001, 512), (15000, 1000), (13000, 1024)])
def test_gradients_of_many_rows_of_few_warps(mb, shape):
    """Rows of one, two and four warps, whose arrays are asked into L2 ahead: every row's gradient, with and without d_sum."""
    import torch
    T, d = shape
    gen = torch.Generator(device="cuda").manual_seed(d)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=gen)
    s, dn, ds, gamma = (t.to(torch.bfloat16) for t in (rand(T, d), rand(T, d), rand(T, d), 1 + 0.2 * rand(d)))
    op = mb.AddRmsNorm(T, d)
    op.forward(s, gamma, n=torch.empty_like(s))
    S, N, G, r = s.double(), dn.double(), gamma.double(), op.rstd.double()[:, None]
    xh, g = S * r, N * G
    ref = r * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    mag = (g.abs() + xh.abs() * (g * xh).abs().mean(dim=1, keepdim=True)) * r
    for d_sum in (ds, None):
        dx, dg = torch.full_like(s, float("nan")), torch.full((d,), float("nan"), device="cuda")
        op.backward(dn, s, gamma, dx, dg, d_sum=d_sum, overwrite=True)
        want = ref if d_sum is None else ref + ds.double()
        assert bool(((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + (d + 11) * U * (mag + ds.double().abs())).all())
        assert bool(((dg.double() - (N * xh).sum(0)).abs() <= (T + 4) * U * (N * xh).abs().sum(0)).all())
