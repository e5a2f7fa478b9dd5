"""Pins of the oracles of the router, the residual norm and the orthogonalised update, and
what their entry points refuse; CPU only."""

import ctypes

import numpy as np
import pytest

from oracle import muon, norm, route

# ------------------------------------------------------------------------ router


def test_route_by_hand():
    l = np.log(np.array([[4.0, 1.0, 2.0, 1.0], [1.0, 1.0, 1.0, 1.0]]))
    ids, w = route.route(l, 2)
    assert ids.tolist() == [[0, 2], [0, 1]]
    np.testing.assert_allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]], rtol=1e-12)
    ids, w = route.route(l, 2, renorm=False, scale=2.0)
    np.testing.assert_allclose(w, [[1.0, 0.5], [0.5, 0.5]], rtol=1e-12)
    # a bias selects, and does not weigh
    ids, w = route.route(l, 2, bias=np.array([0.0, 0.3, 0.0, 0.0]))
    assert ids.tolist() == [[0, 1], [1, 0]]
    np.testing.assert_allclose(w, [[0.8, 0.2], [0.5, 0.5]], rtol=1e-12)
    # sigmoid(log x) = x / (1 + x)
    ids, w = route.route(l, 1, score="sigmoid", renorm=False)
    np.testing.assert_allclose(w, [[0.8], [0.5]], rtol=1e-12)


def test_groups_by_hand():
    # scores 0.9, 0.1 | 0.6, 0.55 | 0.8, 0.05: marks 1.0, 1.15, 0.85
    s = np.array([[0.9, 0.1, 0.6, 0.55, 0.8, 0.05]])
    l = np.log(s / (1 - s))
    assert route.route(l, 2, "sigmoid", groups=3, top_groups=1)[0].tolist() == [[2, 3]]
    assert route.route(l, 3, "sigmoid", groups=3, top_groups=2)[0].tolist() == [[0, 2, 3]]
    # a group of one open expert counts it alone; one of none comes last
    l[0, 3] = -np.inf
    assert route.route(l, 2, "sigmoid", groups=3, top_groups=2)[0].tolist() == [[0, 4]]
    l[0, :4] = -np.inf
    ids, w = route.route(l, 4, "sigmoid", groups=3, top_groups=2)
    assert ids.tolist() == [[4, 5, -1, -1]] and w[0, 2] == w[0, 3] == 0


def test_closed_experts_and_infinities():
    l = np.array([[np.nan, -np.inf, 0.0, np.inf, np.inf], [-np.inf] * 5])
    ids, w = route.route(l, 3, renorm=False)
    assert ids.tolist() == [[3, 4, 2], [-1, -1, -1]]
    np.testing.assert_allclose(w, [[0.5, 0.5, 0.0], [0, 0, 0]])
    assert not route.backward(l, ids, np.ones((2, 3)), renorm=False)[1].any()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(1)
    T, E, k = 4, 7, 3
    l, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    l[0, 2] = -np.inf
    ids, _ = route.route(l, k, score)

    def loss(x):
        total = 0.0
        for t in range(T):
            s = route.scores(x[t], score)[ids[t]]
            total += (dw[t] * 1.5 * (s / (s.sum() + route.TINY) if renorm else s)).sum()
        return total

    got = route.backward(l, ids, dw, score, renorm, 1.5)
    h = 1e-6
    for t, e in np.ndindex(T, E):
        if l[t, e] == -np.inf:
            assert got[t, e] == 0
            continue
        x = l.copy()
        x[t, e] += h
        up = loss(x)
        x[t, e] -= 2 * h
        assert abs((up - loss(x)) / (2 * h) - got[t, e]) < 1e-8


# -------------------------------------------------------------------------- norm

def test_e4m3_values_and_ties():
    values = sorted({(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)} | {m * 2.0 ** -9 for m in range(8)})
    values = [v for v in values if v <= 448]
    np.testing.assert_array_equal(norm.e4m3(np.array(values)), values)
    for i, (a, b) in enumerate(zip(values, values[1:])):
        even = a if i % 2 == 0 else b                       # codes count up with the values
        assert norm.e4m3(np.array([(a + b) / 2]))[0] == even
        assert norm.e4m3(np.array([(a + b) / 2 * (1 + 1e-12)]))[0] == b
    assert norm.e4m3(np.array([460.0, -1e9])).tolist() == [448.0, -448.0]
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).standard_normal(4000).astype(np.float32) * 10
    np.testing.assert_array_equal(norm.e4m3(x.astype(np.float64)), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_norm_by_hand_and_scales():
    s = np.array([[3.0, -4.0, 0.0, 0.0], [0.0] * 4])
    n, codes, scales, r = norm.forward(s, np.ones(4), 0.25 * 4 - 0.25, 0)      # mean 6.25, eps 0.75: r = 1 / sqrt(7)
    np.testing.assert_allclose(r, [7.0 ** -0.5, 0.75 ** -0.5], rtol=1e-12)
    np.testing.assert_allclose(scales[:, 0], [4 / 7 ** 0.5 / 448, 1.0], rtol=1e-7)
    # 3 / 4 of 448 is half way between 320 and 352; the scale is kept in float32, here a little below
    # 4 / (448 sqrt(7)), and so the quotient is above the half
    assert float(np.float32(4 / 7 ** 0.5 / 448)) < 4 / 7 ** 0.5 / 448
    assert codes.tolist() == [[352.0, -448.0, 0.0, 0.0], [0.0] * 4]
    rng = np.random.default_rng(3)
    s = rng.standard_normal((3, 300))
    n, codes, scales, _ = norm.forward(s, np.ones(300), 1e-6, 128)
    assert scales.shape == (3, 3)
    back = codes * np.repeat(scales, 128, axis=1)[:, :300]
    assert np.all(np.abs(back - n) <= np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10 * np.repeat(scales, 128, axis=1)[:, :300]) * (1 + 1e-6))


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(4)
    T, d = 3, 8
    s, g, dn, ds = rng.standard_normal((T, d)), rng.standard_normal(d), rng.standard_normal((T, d)), rng.standard_normal((T, d))
    loss = lambda s, g: (dn * norm.forward(s, g, 1e-6)[0]).sum() + (ds * s).sum()
    dx, dg = norm.backward(dn, s, g, norm.forward(s, g, 1e-6)[3], ds)
    h = 1e-6
    for at, grad, f in ((s, dx, lambda: loss(s, g)), (g, dg, lambda: loss(s, g))):
        for i in np.ndindex(at.shape):
            keep = at[i]
            at[i] = keep + h
            up = f()
            at[i] = keep - h
            down = f()
            at[i] = keep
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


# -------------------------------------------------------------------------- muon

def test_orthogonalize_works_on_the_singular_values():
    rng = np.random.default_rng(5)
    u = rng.standard_normal((5, 8))
    p, s, q = np.linalg.svd(u, full_matrices=False)
    x = s / (np.linalg.norm(s) + 1e-7)
    for a, b, c in (muon.COEFFICIENTS,) * 5:
        x = a * x + b * x ** 3 + c * x ** 5
    np.testing.assert_allclose(muon.orthogonalize(u), p * x @ q, atol=1e-12)
    np.testing.assert_allclose(muon.orthogonalize(u.T), muon.orthogonalize(u).T, atol=1e-12)
    assert np.all((x > 0.6) & (x < 1.25))
    # the cubic whose fixed point is 1 converges to the orthogonal factor
    np.testing.assert_allclose(muon.orthogonalize(u, ((1.5, -0.5, 0.0),) * 40), p @ q, atol=1e-9)
    assert not muon.orthogonalize(np.zeros((3, 4))).any()


def test_muon_step_by_hand():
    w, m, g = np.array([[2.0]]), np.array([[1.0]]), np.array([[3.0]])
    coef = ((1.0, 0.0, 0.0),)                               # X = u / |u|: the sign
    w1, m1 = muon.muon_step(w, m, g, 0.1, 0.5, wd=0.2, scale=2.0, coefficients=coef, eps=0.0)
    assert m1[0, 0] == 3.5 and abs(w1[0, 0] - (2.0 * 0.98 - 0.2)) < 1e-12


# --------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def mb():
    import __graft_entry__
    __graft_entry__.build()
    import mlp_block_backprop_gb300
    return mlp_block_backprop_gb300


def _addresses(n):
    return [0x10000000 * (i + 1) for i in range(n)]  # aligned, never dereferenced


ROUTE = dict(tokens=10, experts=12, top_k=3, score="softmax", groups=4, top_groups=2)


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=1 << 31), dict(experts=0), dict(experts=260), dict(experts=13), dict(top_k=0),
                                dict(top_k=17), dict(top_k=7), dict(groups=0), dict(groups=5), dict(groups=65, experts=130),
                                dict(top_groups=0), dict(top_groups=5), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_route_desc_refusals(mb, kw):
    d = mb.make_route_desc(**{**ROUTE, **kw})
    p = _addresses(4)
    assert mb.lib.mlpblk_moe_route(ctypes.byref(d), *p, None) == mb.MLPBLK_EINVAL
    assert mb.lib.mlpblk_moe_route_backward(ctypes.byref(d), *p, None) == mb.MLPBLK_EINVAL
    with pytest.raises(mb.MlpBlkError):
        mb.MoeRouter(**{**ROUTE, **kw})


def test_route_desc_kinds(mb):
    for field, value in (("score", 2), ("dtype", 7)):
        d = mb.make_route_desc(**ROUTE)
        setattr(d, field, value)
        assert mb.lib.mlpblk_moe_route(ctypes.byref(d), *_addresses(4), None) == mb.MLPBLK_ENOTSUP
    d = mb.make_route_desc(**ROUTE)
    d.renorm = 2
    assert mb.lib.mlpblk_moe_route(ctypes.byref(d), *_addresses(4), None) == mb.MLPBLK_EINVAL
    with pytest.raises(mb.MlpBlkError):
        mb.make_route_desc(**{**ROUTE, "score": "tanh"})
    empty = mb.make_route_desc(**{**ROUTE, "tokens": 0})
    assert mb.lib.mlpblk_moe_route(ctypes.byref(empty), *[None] * 4, None) == mb.MLPBLK_OK
    assert mb.lib.mlpblk_moe_route_backward(ctypes.byref(empty), *[None] * 4, None) == mb.MLPBLK_OK
    mb.MoeRouter(**{**ROUTE, "tokens": 0})


@pytest.mark.parametrize("kw,code", [(dict(tokens=-1), 1), (dict(tokens=1 << 31), 1), (dict(width=0), 1), (dict(width=16385), 2),
                                     (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(block=64), 2)])
def test_norm_desc_refusals(mb, kw, code):
    d = mb.make_norm_desc(**{**dict(tokens=10, width=64), **kw})
    p = _addresses(8)
    assert mb.mlpblk_add_rmsnorm_workspace_size(d) == 0
    assert mb.lib.mlpblk_add_rmsnorm(ctypes.byref(d), *p[:8], None, None) == code
    assert mb.lib.mlpblk_add_rmsnorm_backward(ctypes.byref(d), *p[:7], 0, p[7], 1 << 40, None) == code


def test_norm_argument_refusals(mb):
    d = mb.make_norm_desc(10, 64)
    f = lambda x, res, g, s, n, c, sc, r: mb.lib.mlpblk_add_rmsnorm(ctypes.byref(d), x, res, g, s, n, c, sc, r, None)
    x, res, g, s, n, c, sc, r = _addresses(8)
    for q in ((x, res, g, None, n, c, sc, r), (x, None, g, s, n, c, sc, r), (x, res, g, s, n, c, None, r), (x, res, g, s, n, None, sc, r),
              (x, res, g, s, None, None, None, r), (None, res, g, s, n, c, sc, r), (x, res, None, s, n, c, sc, r)):
        assert f(*q) == mb.MLPBLK_EINVAL
    ws = mb.mlpblk_add_rmsnorm_workspace_size(d)
    b = lambda *a, ow=0, size=ws: mb.lib.mlpblk_add_rmsnorm_backward(ctypes.byref(d), *a[:7], ow, a[7], size, None)
    p = _addresses(8)
    assert b(*p, size=ws - 1) == mb.MLPBLK_EWORKSPACE
    assert b(*p, ow=2) == mb.MLPBLK_EINVAL
    for i in (0, 2, 3, 4, 5, 6, 7):                            # all but d_sum
        q = list(p)
        q[i] = None
        assert b(*q) == mb.MLPBLK_EINVAL, i


def _ortho(mb, **kw):
    return mb.make_ortho_desc(**{**dict(rows=40, cols=50), **kw})


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0), dict(rows=131073), dict(batch=0), dict(batch=65536), dict(eps=-1.0),
                                dict(rows=131072, cols=131072, batch=64), dict(coefficients=(1.0, float("nan"), 0.0))])
def test_ortho_desc_refusals(mb, kw):
    d = _ortho(mb, **kw)
    p = _addresses(6)
    assert mb.mlpblk_orthogonalize_workspace_size(d) == 0
    assert mb.lib.mlpblk_orthogonalize(ctypes.byref(d), *p[:3], 1 << 50, None) == mb.MLPBLK_EINVAL
    hp = mb.Muon(0.1, 0.9, 0.0, 1.0, 1)
    assert mb.lib.mlpblk_muon_step(ctypes.byref(d), ctypes.byref(hp), *p[:4], None, p[4], 1 << 50, None) == mb.MLPBLK_EINVAL
    with pytest.raises(mb.MlpBlkError):
        mb.Orthogonalizer(**{**dict(rows=40, cols=50), **kw}, device="cpu")


def test_ortho_steps_and_coefficients(mb):
    for steps in (0, 17):
        with pytest.raises(mb.MlpBlkError):
            mb.Orthogonalizer(40, 50, steps=steps, device="cpu")
    with pytest.raises(mb.MlpBlkError):
        _ortho(mb, steps=3, coefficients=[(1.0, 0.0, 0.0)] * 2)
    with pytest.raises(mb.MlpBlkError):
        _ortho(mb, steps=1, coefficients=[(1.0, 0.0)])
    d = _ortho(mb, steps=2, coefficients=[(1.0, 2.0, 3.0), (4.0, 5.0, 6.0)])
    assert [list(c) for c in d.coefficients[:2]] == [[1, 2, 3], [4, 5, 6]]
    d.dtype = 9
    assert mb.lib.mlpblk_orthogonalize(ctypes.byref(d), *_addresses(3), 1 << 50, None) == mb.MLPBLK_ENOTSUP
    assert mb.lib.mlpblk_orthogonalize_workspace_size(None) == 0


@pytest.mark.parametrize("hp", [(-0.1, 0.9, 0.0, 1.0, 1), (0.1, 1.0, 0.0, 1.0, 1), (0.1, -0.1, 0.0, 1.0, 1), (0.1, 0.9, -1.0, 1.0, 1),
                                (float("nan"), 0.9, 0.0, 1.0, 1), (0.1, 0.9, 0.0, float("inf"), 1), (0.1, 0.9, 0.0, 1.0, 2)])
def test_muon_hyper_parameters(mb, hp):
    d = _ortho(mb)
    p = _addresses(6)
    assert mb.lib.mlpblk_muon_step(ctypes.byref(d), ctypes.byref(mb.Muon(*hp)), *p[:4], None, p[4], 1 << 50, None) == mb.MLPBLK_EINVAL
    assert mb.lib.mlpblk_muon_step(ctypes.byref(d), None, *p[:4], None, p[4], 1 << 50, None) == mb.MLPBLK_EINVAL


def _spans(mb):
    """Every call with its arguments' sizes in bytes (None: not given), which are outputs, pairs that may be
    the same buffer, and a call of it."""
    at = ctypes.byref
    T, E, k = 37, 12, 3
    r = mb.make_route_desc(T, E, k, dtype="f32")
    yield ("route", [4 * T * E, 4 * E, 4 * T * k, 4 * T * k], (2, 3), (), lambda q: mb.lib.mlpblk_moe_route(at(r), *q, None))
    yield ("route_backward", [4 * T * E, 4 * T * k, 4 * T * k, 4 * T * E], (3,), (), lambda q: mb.lib.mlpblk_moe_route_backward(at(r), *q, None))
    d = 200
    for block, scales in ((0, 1), (128, 2)):
        n = mb.make_norm_desc(T, d, block=block)
        row = 2 * T * d
        yield ("norm", [row, row, 2 * d, row, row, T * d, 4 * T * scales, 4 * T], (3, 4, 5, 6, 7), ((3, 0), (3, 1)),
               lambda q, n=n: mb.lib.mlpblk_add_rmsnorm(at(n), *q, None))
    n = mb.make_norm_desc(T, d)
    ws = mb.mlpblk_add_rmsnorm_workspace_size(n)
    yield ("norm_backward", [row, row, row, 4 * T, 2 * d, row, 4 * d, ws], (5, 6, 7), ((5, 0), (5, 1)),
           lambda q: mb.lib.mlpblk_add_rmsnorm_backward(at(n), *q[:7], 0, q[7], ws, None))
    o = mb.make_ortho_desc(40, 50, 3, dtype="f32")
    N, ws2 = 40 * 50 * 3, mb.mlpblk_orthogonalize_workspace_size(o)
    yield ("orthogonalize", [4 * N, 2 * N, ws2], (1, 2), (), lambda q: mb.lib.mlpblk_orthogonalize(at(o), *q, ws2, None))
    hp = mb.Muon(0.1, 0.9, 0.0, 1.0, 1)
    yield ("muon", [4 * N, 4 * N, 4 * N, 4 * N, 4, ws2], (0, 1, 3, 5), (),
           lambda q: mb.lib.mlpblk_muon_step(at(o), at(hp), *q, ws2, None))


def test_outputs_that_share_bytes_are_refused(mb):
    """Each output laid over the beginning, the end and the middle of every other argument.  (No call
    here would be accepted: the addresses are never used.)"""
    for name, sizes, outs, same, call in _spans(mb):
        base = [0x100000000 * (i + 1) for i in range(len(sizes))]
        for o in outs:
            for i in range(len(sizes)):
                if i == o:
                    continue
                inside = (sizes[i] - 1) // 16 * 16
                for at in (base[i], base[i] + inside, base[i] - (sizes[o] - 1) // 16 * 16, base[i] + inside // 32 * 16):
                    if ((o, i) in same or (i, o) in same) and at == base[i]:
                        continue
                    q = list(base)
                    q[o] = at
                    assert call(q) == mb.MLPBLK_EINVAL, (name, "argument", o, "over", i, hex(at))


def test_misaligned_pointers_are_refused(mb):
    for name, sizes, outs, same, call in _spans(mb):
        for i in range(len(sizes)):
            q = [0x100000000 * (j + 1) for j in range(len(sizes))]
            q[i] += 2 if (name, i) == ("muon", 4) else 8
            assert call(q) == mb.MLPBLK_EINVAL, (name, i)


def test_workspace_sizes(mb):
    d = _ortho(mb, rows=300, cols=200, batch=2)
    need = mb.mlpblk_orthogonalize_workspace_size(d)
    # three X of whole lines, four square matrices
    assert need >= 2 * (3 * 300 * 256 + 4 * 200 * 256) * 2
    assert mb.lib.mlpblk_orthogonalize(ctypes.byref(d), *_addresses(3), need - 1, None) == mb.MLPBLK_EWORKSPACE
    hp = mb.Muon(0.1, 0.9, 0.0, 1.0, 1)
    p = _addresses(6)
    assert mb.lib.mlpblk_muon_step(ctypes.byref(d), ctypes.byref(hp), *p[:4], None, p[4], need - 1, None) == mb.MLPBLK_EWORKSPACE
    assert mb.mlpblk_add_rmsnorm_workspace_size(mb.make_norm_desc(5, 100)) == 5 * 128 * 4
    assert mb.mlpblk_add_rmsnorm_workspace_size(mb.make_norm_desc(1 << 20, 100)) == 1024 * 128 * 4


def test_binding_refuses_wrong_tensors(mb):
    torch = pytest.importorskip("torch")
    r = mb.MoeRouter(4, 8, 2, dtype="f32")
    r._t.device = lambda: 0
    try:
        with pytest.raises(mb.MlpBlkError):                   # not on the GPU
            r.route(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
        with pytest.raises(mb.MlpBlkError):
            r.route_backward(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), torch.zeros(4, 8))
    finally:
        mb._Torch._one = None
    with pytest.raises(mb.MlpBlkError):
        mb.AddRmsNorm(4, 20000, device="cpu")
    with pytest.raises(mb.MlpBlkError):
        mb.make_norm_desc(4, 8, dtype="f16")


def test_both_ways_into_the_library_agree(mb):
    slow = {n: mb._Calls._ctypes("mlpblk_" + n) for n in ("moe_route", "moe_route_backward", "add_rmsnorm", "add_rmsnorm_backward", "orthogonalize")}
    at = ctypes.addressof
    r, n, o = mb.make_route_desc(**ROUTE), mb.make_norm_desc(10, 64), _ortho(mb)
    a = _addresses(8)
    cases = [("moe_route", (at(r), a[0], None, a[0], a[1], None)), ("moe_route_backward", (at(r), a[0], a[1], a[2], a[0], None)),
             ("add_rmsnorm", (at(n), a[0], None, a[1], None, None, None, None, a[2], None)),
             ("add_rmsnorm_backward", (at(n), a[0], None, a[1], a[2], a[3], a[4], a[5], 0, a[6], 3, None)),
             ("orthogonalize", (at(o), a[0], a[1], a[2], 5, None))]
    for name, args in cases:
        rc = slow[name](*args)
        assert rc in (mb.MLPBLK_EINVAL, mb.MLPBLK_EWORKSPACE)
        assert getattr(mb._calls, name)(*args) == rc, name


def test_version_tells_of_the_operators(mb):
    assert mb.mlpblk_version() >= 102
