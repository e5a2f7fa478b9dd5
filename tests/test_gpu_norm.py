"""The residual sum with RMSNorm and E4M3 codes against the oracle (oracle.norm), GB300 only.

The sum, codes and scales are compared exactly, rstd to its last bit.  n in the tensors'
type: three roundings of 2^-24 and half a step of the type (bf16 2^-8).  dx: the row's dot
product is a sum of `width` float32 terms ((width + 3) * 2^-24 of their magnitudes), each of
the three summands has up to six more roundings, the result half a step of its type.
dgamma: tokens + 4 roundings of 2^-24 of its terms' magnitudes.
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


def _guarded(n, dtype):
    """A tensor of n elements between two bands that nothing may touch."""
    import torch
    whole = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda").repeat(torch.empty((), dtype=dtype).element_size()).view(dtype)
    return whole[128:128 + n], whole


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 127), (9, 128), (4, 129), (7, 256), (300, 264), (33, 1000), (70, 1001), (11, 2048),
          (200, 2049), (1300, 1024), (17, 4096), (900, 4096), (5, 5003), (40, 8192), (3, 10001), (200, 12288), (161, 16384), (20, 16383)]


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(mb, shape, dtype, block):
    import torch
    T, d = shape
    rng = np.random.default_rng(T + d)
    x, res = _t(rng.normal(0, 1, (T, d)) * np.exp(rng.normal(0, 2, (T, 1))), dtype), _t(rng.normal(0, 1, (T, d)), dtype)
    gamma = _t(1 + rng.normal(0, 0.2, d), dtype)
    x[T // 2] = 0          # a row of zeros under a zero branch: no scale to find
    res[T // 2] = 0
    for with_res in (True, False):
        op = mb.AddRmsNorm(T, d, 1e-6, dtype, block)
        codes, whole = _guarded(T * d, torch.uint8)
        scales, whole_s = _guarded(T * ((d + 127) // 128 if block else 1), torch.float32)
        n, whole_n = _guarded(T * d, x.dtype)
        s = torch.empty_like(x) if with_res else None
        op.forward(x, gamma, codes.view(torch.float8_e4m3fn), scales, n, res if with_res else None, s)
        kept = (x.float() + res.float()).to(x.dtype) if with_res else x
        if with_res:
            assert torch.equal(s, kept)
        ref_n, ref_codes, ref_scales, ref_r = norm.forward(to_np(kept), to_np(gamma), 1e-6, block)
        np.testing.assert_array_equal(to_np(scales).reshape(T, -1), ref_scales.astype(np.float64))
        np.testing.assert_array_equal(to_np(codes.view(torch.float8_e4m3fn)).reshape(T, d), ref_codes)
        np.testing.assert_allclose(to_np(op.rstd), ref_r, rtol=2.0 ** -23)
        half = 2.0 ** -8 if dtype == "bf16" else U
        np.testing.assert_allclose(to_np(n).reshape(T, d), ref_n, rtol=3 * U + half, atol=1e-37)
        for w in (whole, whole_s, whole_n):
            b = w.view(torch.uint8)
            e = 128 * w.element_size()
            assert bool((b[:e] == 77).all()) and bool((b[-e:] == 77).all())
        # without the optional outputs the others are the same
        codes2, scales2 = torch.empty_like(codes), torch.empty_like(scales)
        desc = mb.make_norm_desc(T, d, 1e-6, dtype, block)
        mb.mlpblk_add_rmsnorm(desc, x, res if with_res else None, gamma, s, None, codes2, scales2, None)
        assert torch.equal(codes2, codes) and torch.equal(scales2, scales)
        n2 = torch.empty_like(n)
        mb.mlpblk_add_rmsnorm(desc, x, res if with_res else None, gamma, s, n2, None, None, None)
        assert torch.equal(n2, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(mb, shape, dtype):
    import torch
    T, d = shape
    rng = np.random.default_rng(T * 3 + d)
    s, dn, ds = (_t(rng.normal(0, 1, (T, d)), dtype) for _ in range(3))
    gamma = _t(1 + rng.normal(0, 0.2, d), dtype)
    op = mb.AddRmsNorm(T, d, 1e-6, dtype)
    op.forward(s, gamma, n=torch.empty_like(s))
    r = to_np(op.rstd)
    start = torch.from_numpy(rng.normal(0, 1, d).astype(np.float32)).cuda()
    half = 2.0 ** -8 if dtype == "bf16" else U
    S, N, G, D = to_np(s), to_np(dn), to_np(gamma), to_np(ds)
    for with_sum in (True, False):
        dx, dg = torch.full_like(s, float("nan")), start.clone()
        op.backward(dn, s, gamma, dx, dg, d_sum=ds if with_sum else None)
        ref_dx, ref_dg = norm.backward(N, S, G, r, D if with_sum else None)
        dots = (np.abs(N * G * S)).sum(axis=1, keepdims=True) / d
        mag = np.abs(N * G) * r[:, None] + np.abs(S) * r[:, None] ** 3 * dots
        tol = half * np.abs(ref_dx) + 8 * U * (mag + np.abs(D)) + (d + 3) * U * np.abs(S) * r[:, None] ** 3 * dots
        err = np.abs(to_np(dx) - ref_dx)
        assert np.all(err <= tol), (err - tol).max()
        mag = np.abs(N * S * r[:, None]).sum(axis=0)
        err = np.abs(to_np(dg) - (to_np(start) + ref_dg))
        assert np.all(err <= (T + 4) * U * (mag + np.abs(to_np(start)))), err.max()
    # set instead of added to, over NaN; dx in the place of either gradient: the same bits
    dg2 = torch.full_like(start, float("nan"))
    op.backward(dn, s, gamma, dx, dg2, overwrite=True)
    zero = torch.zeros_like(start)
    op.backward(dn, s, gamma, dx, zero)
    assert torch.equal(dg2, zero)
    want = torch.empty_like(s)
    op.backward(dn, s, gamma, want, dg2, d_sum=ds, overwrite=True)
    for which in (0, 1):
        a, b = dn.clone(), ds.clone()
        op.backward(a, s, gamma, (a, b)[which], dg2, d_sum=b, overwrite=True)
        assert torch.equal((a, b)[which], want) and torch.equal(dg2, zero)


def test_gradients_against_differences(mb):
    """Central differences of L = sum dn n + sum d_sum s in float32."""
    import torch
    T, d = 3, 40
    rng = np.random.default_rng(2)
    s, dn, ds = (torch.from_numpy(rng.normal(0, 1, (T, d)).astype(np.float32)).cuda() for _ in range(3))
    gamma = torch.from_numpy((1 + rng.normal(0, 0.2, d)).astype(np.float32)).cuda()
    op = mb.AddRmsNorm(T, d, 1e-6, "f32")
    n = torch.empty_like(s)

    def loss(x, g):
        op.forward(x, g, n=n)
        return float((dn.double() * n.double()).sum() + (ds.double() * x.double()).sum())

    loss(s, gamma)
    dx, dg = torch.empty_like(s), torch.empty(d, device="cuda")
    op.backward(dn, s, gamma, dx, dg, d_sum=ds, overwrite=True)
    h = 2.0 ** -6
    # L is a sum of T d products below 10 whose n is off by 4 roundings; third derivatives below 60
    bound = 60 * h * h + T * d * 10 * 4 * U / h
    for t, c in ((0, 0), (1, 17), (2, 39)):
        x = s.clone()
        x[t, c] += h
        up = loss(x, gamma)
        x[t, c] -= 2 * h
        assert abs((up - loss(x, gamma)) / (2 * h) - float(dx[t, c])) <= bound
    for c in (0, 20, 39):
        g = gamma.clone()
        g[c] += h
        up = loss(s, g)
        g[c] -= 2 * h
        assert abs((up - loss(s, g)) / (2 * h) - float(dg[c])) <= bound


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
def test_values_at_the_edges(mb, dtype, block):
    """Halves between two codes, tiny and huge rows, infinities and NaN."""
    import torch
    d = 512
    rows = np.ones((8, d))
    rows[0, :16] = 448.0 * 2.0 ** -np.arange(16)     # codes down to E4M3's smallest and below
    rows[1] = (np.arange(d) % 61 + 1) / 32.0         # short ratios: many halves
    rows[2] = 1e-30
    rows[3] = 1e15
    rows[4, 300] = np.inf
    rows[5, 10] = np.nan
    rows[6] = 0.0
    rows[7, ::2] = -1e-38
    x, gamma = _t(rows, dtype), _t(np.where(np.arange(d) % 7 == 0, 1.5, 1.0), dtype)
    op = mb.AddRmsNorm(8, d, 1e-6, dtype, block)
    codes = torch.empty(8, d, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(8, 4 if block else 1, device="cuda")
    op.forward(x, gamma, codes, scales)
    fine = [0, 1, 2, 3, 6, 7]
    _, ref_codes, ref_scales, ref_r = norm.forward(to_np(x)[fine], to_np(gamma), 1e-6, block)
    np.testing.assert_array_equal(to_np(scales)[fine], ref_scales.astype(np.float64))
    np.testing.assert_array_equal(to_np(codes)[fine], ref_codes)
    np.testing.assert_allclose(to_np(op.rstd)[fine], ref_r, rtol=2.0 ** -23)
    for t in (4, 5):
        assert np.isnan(to_np(op.rstd)[t]) and np.isnan(to_np(scales)[t]).all() and np.isnan(to_np(codes)[t]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
def test_products_beyond_the_range(mb, dtype, block):
    """sum * gamma overflows in one column: its scale is NaN, rstd is not."""
    import torch
    T, d = 5, 300
    rng = np.random.default_rng(6)
    x, gamma = _t(rng.normal(0, 1, (T, d)), dtype), _t(np.ones(d), dtype)
    x[3, 200], gamma[200] = 2.0 ** 20, 2.0 ** 110
    op = mb.AddRmsNorm(T, d, 1e-6, dtype, block)
    per = 3 if block else 1
    codes, scales = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, per, device="cuda")
    op.forward(x, gamma, codes, scales)
    _, ref_codes, ref_scales, ref_r = norm.forward(to_np(x), to_np(gamma), 1e-6, block)
    np.testing.assert_allclose(to_np(op.rstd), ref_r, rtol=2.0 ** -23)
    bad = np.zeros((T, per), dtype=bool)
    bad[3, 1 if block else 0] = True
    got = to_np(codes.view(torch.float8_e4m3fn))
    wide = np.repeat(bad, 128 if block else d, axis=1)[:, :d]
    assert np.isnan(to_np(scales)[bad]).all() and np.isnan(got[wide]).all()
    np.testing.assert_array_equal(to_np(scales)[~bad], ref_scales.astype(np.float64)[~bad])
    np.testing.assert_array_equal(got[~wide], ref_codes[~wide])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sum_in_place(mb, dtype):
    """The residual stream updated where it lies, and x likewise."""
    import torch
    T, d = 333, 1001
    rng = np.random.default_rng(9)
    x, res, gamma = _t(rng.normal(0, 1, (T, d)), dtype), _t(rng.normal(0, 1, (T, d)), dtype), _t(np.ones(d), dtype)
    op = mb.AddRmsNorm(T, d, dtype=dtype)
    want, n = torch.empty_like(x), torch.empty_like(x)
    op.forward(x, gamma, n=n, residual=res, sum=want)
    for which in (0, 1):
        a, b, m = x.clone(), res.clone(), torch.empty_like(x)
        op.forward(a, gamma, n=m, residual=b, sum=(a, b)[which])
        assert torch.equal((a, b)[which], want) and torch.equal((b, a)[which], (res, x)[which]) and torch.equal(m, n)


def test_capture_and_replay(mb):
    import torch
    T, d = 700, 1024
    rng = np.random.default_rng(4)
    x, dn = _t(rng.normal(0, 1, (T, d)), "bf16"), _t(rng.normal(0, 1, (T, d)), "bf16")
    gamma = _t(np.ones(d), "bf16")
    op = mb.AddRmsNorm(T, d)
    codes, scales = torch.empty(T, d, dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda")
    dx, dg = torch.empty_like(x), torch.empty(d, device="cuda")

    def run():
        op.forward(x, gamma, codes, scales)
        op.backward(dn, x, gamma, dx, dg, overwrite=True)

    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    x.copy_(_t(rng.normal(0, 2, (T, d)), "bf16"))
    g.replay()
    got = [t.clone() for t in (codes, scales, dx, dg)]
    run()
    assert all(torch.equal(a, b) for a, b in zip(got, (codes, scales, dx, dg)))


def test_no_tokens(mb):
    import torch
    op = mb.AddRmsNorm(0, 64)
    e, dg = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.full((64,), 3.0, device="cuda")
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    op.forward(e, gamma, n=e)
    op.backward(e, e, gamma, e, dg)
    assert bool((dg == 3).all())
    op.backward(e, e, gamma, e, dg, overwrite=True)
    assert not dg.any()


@pytest.mark.parametrize("block", [0, 128])
def test_offsets_beyond_32_bits(mb, block):
    """2^32 values and more: the last rows against the oracle, and their gradient."""
    import torch
    T, d, last = (1 << 20) + 37, 4104, 6
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_()
    gamma = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    per = (d + 127) // 128 if block else 1
    codes, scales = torch.zeros(T, d, dtype=torch.uint8, device="cuda"), torch.zeros(T, per, device="cuda")
    op = mb.AddRmsNorm(T, d, 1e-6, "bf16", block)
    op.forward(x, gamma, codes, scales)
    dx, dg = torch.zeros_like(x), torch.zeros(d, device="cuda")
    op.backward(x, x, gamma, dx, dg, overwrite=True)
    n = T - last
    X = to_np(x[n:])
    _, ref_codes, ref_scales, r = norm.forward(X, np.ones(d), 1e-6, block)
    np.testing.assert_array_equal(to_np(scales[n:]).reshape(last, -1), ref_scales.astype(np.float64))
    np.testing.assert_array_equal(to_np(codes[n:].view(torch.float8_e4m3fn)), ref_codes)
    ref, _ = norm.backward(X, X, np.ones(d), r)
    # dx = r x (1 - r^2 mean x^2) cancels to next to nothing: (d + 12) roundings of r x
    assert np.all(np.abs(to_np(dx[n:]) - ref) <= 2.0 ** -8 * np.abs(ref) + (d + 12) * U * np.abs(X) * r[:, None])
    # dgamma_k = sum_t x^2 r: T terms near 1, each CTA's share in order, then a tree
    assert bool(((dg / T - 1).abs() < 0.01).all())
