"""A training step of routed experts through the operators one after another: residual norm,
router, sort, experts at 4 bits, weighted sum; the gradients back to the residual stream, gamma and the
router's weight; Muon on the experts' weights.  Each stage against its oracle on the stage's own
input, at the tolerances of that stage's own tests; eager, then captured and replayed on other inputs.
GB300 only."""

import numpy as np
import pytest

from oracle import fp4, muon, norm, route, sort
from helpers import to_np

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def mb():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mlp_block_backprop_gb300 as mb
    yield mb
    assert mb.mlpblk_last_error() == mb.MLPBLK_OK


def test_routed_step(mb):
    import torch
    T, d, E, k, G, TG, pad = 210, 96, 16, 3, 4, 2, 256
    bf, dev = torch.bfloat16, dict(device="cuda")
    rng = np.random.default_rng(31)
    fill = lambda t, std=1.0: t.copy_(torch.from_numpy((rng.standard_normal(tuple(t.shape)) * std).astype(np.float32)))
    x, res, dy = (torch.zeros(T, d, dtype=bf, **dev) for _ in range(3))
    gamma, wr, bias = torch.zeros(d, dtype=bf, **dev), torch.zeros(E, d, dtype=bf, **dev), torch.zeros(E, **dev)
    w = torch.zeros(E, d, d, **dev)                     # the experts: one matrix each (float32 masters)
    wb, m = torch.zeros(E, d, d, dtype=bf, **dev), torch.zeros(E, d, d, **dev)
    # the handles and buffers that a program keeps
    nm, rt, s = mb.AddRmsNorm(T, d), mb.MoeRouter(T, E, k, "sigmoid", G, TG, True, 1.5), mb.MoeSort(T, d, E, k, pad)
    R = s.rows
    wq, wtq, nq = mb.Fp4Matrix(d, d, batch=E), mb.Fp4Matrix(d, d, batch=E), mb.Fp4Matrix(R, d)
    dq, dtq, ntq = mb.Fp4Matrix(R, d), mb.Fp4Matrix(d, R), mb.Fp4Matrix(d, R)
    opt = mb.Orthogonalizer(d, d, batch=E, dtype="bf16")
    n, sum_, rows, d_rows, dn_rows = (torch.zeros(r, d, dtype=bf, **dev) for r in (T, T, R, R, R))
    codes, scales = torch.zeros(T, d, dtype=torch.float8_e4m3fn, **dev), torch.zeros(T, **dev)
    ids, p, dp = torch.zeros(T, k, dtype=torch.int32, **dev), torch.zeros(T, k, **dev), torch.zeros(T, k, **dev)
    logits, d_logits, y, dn, dx = (torch.zeros(T, c, dtype=bf, **dev) for c in (E, E, d, d, d))
    dg, dw = torch.zeros(d, **dev), torch.zeros(E, d, d, **dev)

    def step():
        nm.forward(x, gamma, codes, scales, n=n, residual=res, sum=sum_)
        torch.mm(n, wr.t(), out=logits)
        rt.route(logits, ids, p, bias=bias)
        s.sort(ids)
        wq.quantize(wb)
        nq.quantize(n, sort=s, gather=True)
        nq.matmul_grouped(wq, s, rows)
        s.unpermute(rows, y, weights=p, residual=sum_)
        # back
        s.unpermute_backward(dy, rows, p, d_rows, dp)
        rt.route_backward(logits, ids, dp, d_logits)
        dq.quantize(d_rows, sort=s)
        wtq.quantize(wb, transposed=True)
        dq.matmul_grouped(wtq, s, dn_rows)
        dtq.quantize(d_rows, sort=s, transposed=True)
        ntq.quantize(n, sort=s, gather=True, transposed=True)
        dtq.wgrad_grouped(ntq, s, dw)
        s.permute_backward(dn_rows, dn)
        dn.add_(d_logits @ wr)
        nm.backward(dn, sum_, gamma, dx, dg, d_sum=dy, overwrite=True)
        opt.muon_step(w, dw, m, 0.02, weight_decay=0.1, scale=0.2 * d ** 0.5, weight=wb)

    def inputs():
        for t in (x, res):
            fill(t)
        fill(dy, 1e-2)
        fill(gamma, 0.1).add_(1.0)
        fill(wr, d ** -0.5)
        fill(bias, 0.05)
        fill(w, d ** -0.5)
        fill(m, 1e-3)
        wb.copy_(w)

    def check(before):
        w0, m0, wb0 = before
        S = to_np(sum_)
        assert torch.equal(sum_, (x.float() + res.float()).to(bf))
        rn, rc, rs, rr = norm.forward(S, to_np(gamma), 1e-6)
        np.testing.assert_array_equal(to_np(scales), rs[:, 0].astype(np.float64))
        np.testing.assert_array_equal(to_np(codes), rc)
        np.testing.assert_allclose(to_np(n), rn, rtol=3 * U + HALF, atol=1e-37)
        l = to_np(logits)
        ri, rw = route.route(l, k, "sigmoid", to_np(bias), G, TG, True, 1.5)
        np.testing.assert_array_equal(ids.cpu().numpy(), ri)
        rtol = (2 * (l.max() - l.min() + 2 + E + 2) + k + 3) * U
        np.testing.assert_allclose(to_np(p), rw, rtol=rtol)
        count, seg, pos, row_map = sort.plan(ri, E, pad)
        np.testing.assert_array_equal(s.pos.cpu().numpy(), pos)
        live = (row_map >= 0)[:, None]
        own = lambda t: np.where(live, to_np(t), 0.0)
        av, bv, dr = np.where(live, to_np(n)[np.maximum(row_map, 0) // k], 0.0), to_np(wb0), own(d_rows)
        a, da = fp4.rounded(av), fp4.rounded(dr)
        at, dat = fp4.rounded(av.T), fp4.rounded(dr.T)

        def product(got, a, b, half=HALF):
            ref, mag = fp4.product(a, b)
            assert np.all(np.abs(got - ref) <= (-(-a.shape[1] // 32) + 2) * 2 * U * mag + half * np.abs(ref))

        for e in range(E):
            r = slice(seg[e], seg[e] + count[e])
            product(to_np(rows)[r], a[r], fp4.rounded(bv[e]))
            product(to_np(dn_rows)[r], da[r], fp4.rounded(bv[e].T))
            r = slice(seg[e], seg[e + 1])
            product(to_np(dw)[e], dat[:, r], at[:, r], 0.0)
        ref, mag = sort.unpermute(own(rows), pos, to_np(p), S)
        assert np.all(np.abs(to_np(y) - ref) <= HALF * np.abs(ref) + (k + 2) * U * mag)
        rdr, rdp, mag = sort.unpermute_backward(to_np(dy), own(rows), pos, row_map, to_np(p))
        assert np.all(np.abs(to_np(dp) - rdp) <= (d + 1) * U * mag)
        rdl = route.backward(l, ri, to_np(dp), "sigmoid", True, 1.5)
        mag = np.zeros((T, E))
        for t in range(T):
            sc, g = route.scores(l[t], "sigmoid")[ri[t]], np.abs(1.5 * to_np(dp)[t])
            mag[t, ri[t]] = (g + (g * sc).sum() / sc.sum()) / sc.sum() * sc
        assert np.all(np.abs(to_np(d_logits) - rdl) <= 4 * rtol * mag + HALF * np.abs(rdl))
        rdx, rdg = norm.backward(to_np(dn), S, to_np(gamma), to_np(nm.rstd), to_np(dy))
        r, N, D = to_np(nm.rstd)[:, None], to_np(dn), to_np(dy)
        dots = np.abs(N * to_np(gamma) * S).sum(axis=1, keepdims=True) / d
        mag = np.abs(N * to_np(gamma)) * r + np.abs(S) * r ** 3 * dots
        assert np.all(np.abs(to_np(dx) - rdx) <= HALF * np.abs(rdx) + 8 * U * (mag + np.abs(D)) + (d + 3) * U * np.abs(S) * r ** 3 * dots)
        assert np.all(np.abs(to_np(dg) - rdg) <= (T + 4) * U * np.abs(N * S * r).sum(axis=0))
        # an expert that nobody chose has no gradient; its weight still follows its momentum
        lr, scale = 0.02, 0.2 * d ** 0.5
        for e in range(E):
            W, M = muon.muon_step(w0[e], m0[e], to_np(dw)[e], lr, 0.95, 0.1, scale)
            assert np.linalg.norm(to_np(m)[e] - M) <= (4 * U + 1e-8) * np.linalg.norm(M) + 2 * U * np.linalg.norm(to_np(dw)[e])
            X = (w0[e] * (1 - lr * 0.1) - W) / (lr * scale)
            assert np.linalg.norm(to_np(w)[e] - W) <= lr * scale * 3e-3 * np.linalg.norm(X) + 4 * U * np.linalg.norm(W)
        assert torch.equal(wb, w.to(bf))

    g = torch.cuda.CUDAGraph()
    for turn in range(4):
        inputs()
        before = to_np(w), to_np(m), wb.clone()
        torch.cuda.synchronize()
        if turn == 1:
            with torch.cuda.graph(g):
                step()
        g.replay() if turn else step()
        torch.cuda.synchronize()
        check(before)
