"""Tokens sorted by expert and back against the oracle (oracle.sort), GB300 only.

The plan and permute are exact.  Tolerances: a sum of n float32 terms is off by at
most (n + 1) * 2^-24 of the terms' magnitudes (a product and an addition each round
once, half a step of 2^-23), a bf16 result by half a step more, 2^-8 of its value
(float32: in the sum already).
"""

import numpy as np
import pytest

from oracle import sort
from helpers import to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mb():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mlp_block_backprop_gb300 as mb
    yield mb
    assert mb.mlpblk_last_error() == mb.MLPBLK_OK


def _ids(rng, T, E, k, kind):
    if kind == "one":
        return np.full((T, k), E - 1, dtype=np.int32)          # every slot the last expert
    if kind == "none":
        return np.where(rng.random((T, k)) < 0.5, -1, E).astype(np.int32)
    idx = rng.integers(0, E, (T, k))
    if kind == "mixed":
        idx = np.where(rng.random((T, k)) < 0.1, rng.choice([-5, E, 1 << 30], (T, k)), idx)
        idx[rng.random((T, k)) < 0.5] = 0
    return idx.astype(np.int32)


def _plan(mb, idx, width, E, pad, dtype="bf16"):
    import torch
    T, k = idx.shape
    s = mb.MoeSort(T, width, E, k, pad, dtype)
    for t in (s.count, s.seg, s.pos, s.row_map):
        t.fill_(77)
    s.sort(torch.from_numpy(idx).cuda())
    return s


@pytest.mark.parametrize("kind", ["any", "one", "none", "mixed"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (1, 256, 8, 128), (33, 7, 3, 16), (500, 256, 8, 256), (513, 60, 8, 1),
                                   (4097, 3, 1, 1024), (5000, 130, 2, 100), (20011, 17, 6, 128), (70001, 40, 2, 16)])
def test_plan(mb, shape, kind):
    T, E, k, pad = shape
    idx = _ids(np.random.default_rng(T), T, E, k, kind)
    s = _plan(mb, idx, 8, E, pad)
    for got, ref in zip((s.count, s.seg, s.pos, s.row_map), sort.plan(idx, E, pad)):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)


def test_plan_of_no_tokens(mb):
    s = _plan(mb, np.zeros((0, 2), dtype=np.int32), 8, 5, 128)
    assert not s.count.any() and not s.seg.any() and s.rows == 0


# widths of 16-, 4- and 2-byte accesses (bf16) and of 16- and 4-byte ones (float32)
MOVES = [(1, 8, 2, 1, 1), (5, 1, 3, 2, 4), (37, 1002, 5, 3, 16), (64, 1001, 4, 6, 1), (130, 4096, 8, 2, 128),
         (9, 5000, 3, 9, 8), (300, 64, 60, 4, 128), (17, 12288, 2, 2, 2),
         # few tokens, whose rows are shared by CTAs, and much padding
         (20, 3051, 85, 7, 128), (3, 20001, 200, 7, 256), (1, 4097, 4, 4, 1024), (151, 9002, 4, 5, 3),
         # the smallest rows
         (1, 1, 1, 1, 1), (3, 1, 2, 2, 1), (2, 3, 2, 1, 1), (7, 5, 3, 2, 2),
         # many tokens, long rows, many slots
         (1300, 1024, 6, 2, 16), (1250, 1027, 5, 6, 1), (700, 6001, 3, 3, 4), (1300, 520, 20, 15, 1), (1300, 1040, 20, 16, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", MOVES)
def test_moves_and_gradients(mb, shape, dtype):
    import torch
    T, d, E, k, pad = shape
    rng = np.random.default_rng(T + d)
    idx = _ids(rng, T, E, k, "mixed")
    s = _plan(mb, idx, d, E, pad, dtype)
    count, seg, pos, row_map = sort.plan(idx, E, pad)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    new = lambda r: torch.from_numpy(rng.standard_normal((r, d)).astype(np.float32)).cuda().to(dt)
    x, dy, rows, g = new(T), new(T), new(s.rows), new(s.rows)
    w = torch.from_numpy(rng.uniform(-1, 1, (T, k)).astype(np.float32)).cuda()
    live, behind = row_map >= 0, np.arange(s.rows) >= seg[E]
    xn, dyn, rn, gn, wn = (to_np(t) for t in (x, dy, rows, g, w))
    # what no entry owns holds NaN: it must not reach an output
    nan = torch.from_numpy(~live).cuda()
    rows[nan], g[nan] = float("nan"), float("nan")
    rn, gn = np.where(live[:, None], rn, 0.0), np.where(live[:, None], gn, 0.0)

    out = torch.full((s.rows, d), 7.0, dtype=dt, device="cuda")
    s.permute(x, out)
    got = to_np(out)
    np.testing.assert_array_equal(got[~behind], sort.permute(xn, row_map, k)[~behind])
    assert np.all(got[behind] == 7.0)

    y = torch.full((T, d), 7.0, dtype=dt, device="cuda")
    for weights, residual in ((w, x), (w, None), (None, x), (None, None)):
        s.unpermute(rows, y, weights=weights, residual=residual)
        ref, mag = sort.unpermute(rn, pos, None if weights is None else wn, None if residual is None else xn)
        assert np.all(np.abs(to_np(y) - ref) <= half * np.abs(ref) + (k + 2) * 2.0 ** -24 * mag)
    y2 = x.clone()
    s.unpermute(rows, y2, weights=w, residual=y2)           # in place on the residual
    s.unpermute(rows, y, weights=w, residual=x)
    assert torch.equal(y2, y)

    dx = torch.full((T, d), 7.0, dtype=dt, device="cuda")
    s.permute_backward(g, dx)
    ref, mag = sort.unpermute(gn, pos)
    np.testing.assert_allclose(ref, sort.permute_backward(gn, pos), rtol=0, atol=1e-12)
    assert np.all(np.abs(to_np(dx) - ref) <= half * np.abs(ref) + (k + 1) * 2.0 ** -24 * mag)

    for weights in (w, None):
        dr = torch.full((s.rows, d), 7.0, dtype=dt, device="cuda")
        dw = torch.full((T, k), 7.0, device="cuda")
        s.unpermute_backward(dy, rows, weights, dr, dw)
        r_dr, r_dw, mag = sort.unpermute_backward(dyn, rn, pos, row_map, None if weights is None else wn)
        got = to_np(dr)
        assert np.all(np.abs(got - r_dr)[~behind] <= (half + 2.0 ** -24) * np.abs(r_dr[~behind]))
        assert np.all(got[behind] == 7.0)
        assert np.all(np.abs(to_np(dw) - r_dw) <= (d + 1) * 2.0 ** -24 * mag)
        assert np.all(to_np(dw)[pos < 0] == 0.0)
        dr2 = torch.zeros(s.rows, d, dtype=dt, device="cuda")
        mb.mlpblk_moe_unpermute_backward(s.desc, dy, None, s.pos, s.count, s.seg, weights, dr2, None)
        assert np.array_equal(to_np(dr2)[~behind], got[~behind])


def test_repeats_are_bitwise_equal(mb):
    import torch
    rng = np.random.default_rng(1)
    idx = _ids(rng, 3000, 16, 4, "any")
    s = _plan(mb, idx, 512, 16, 128)
    dy = torch.randn(3000, 512, device="cuda", dtype=torch.bfloat16)
    rows = torch.randn(s.rows, 512, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(3000, 4, device="cuda")
    first = None
    for _ in range(3):
        dr, dw, y = torch.zeros_like(rows), torch.empty_like(w), torch.empty_like(dy)
        s.unpermute_backward(dy, rows, w, dr, dw)
        s.unpermute(rows, y, weights=w)
        if first is None:
            first = (dr, dw, y)
        assert all(torch.equal(a, b) for a, b in zip(first, (dr, dw, y)))


def test_graph_replay_on_new_ids(mb):
    import torch
    T, d, E, k, pad = 200, 96, 9, 2, 16
    rng = np.random.default_rng(2)
    idx = torch.from_numpy(_ids(rng, T, E, k, "any")).cuda()
    s = mb.MoeSort(T, d, E, k, pad)
    x = torch.randn(T, d, device="cuda").to(torch.bfloat16)
    rows, y = torch.zeros(s.rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.sort(idx)
        s.permute(x, rows)
        s.unpermute(rows, y)
    for seed in (3, 4):
        new = _ids(np.random.default_rng(seed), T, E, k, "mixed")
        idx.copy_(torch.from_numpy(new))
        x.normal_()
        g.replay()
        torch.cuda.synchronize()
        count, seg, pos, row_map = sort.plan(new, E, pad)
        np.testing.assert_array_equal(s.pos.cpu().numpy(), pos)
        ref, mag = sort.unpermute(sort.permute(to_np(x), row_map, k), pos)
        assert np.all(np.abs(to_np(y) - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -24 * mag)


def test_binding_checks(mb):
    import torch
    s = mb.MoeSort(4, 8, 3, 2, 16)
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (idx.long(), idx.cpu(), idx[:3], torch.zeros(4, 4, dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(mb.MlpBlkError):
            s.sort(bad)
    with pytest.raises(mb.MlpBlkError):
        s.permute(torch.zeros(4, 8, device="cuda"), torch.zeros(s.rows, 8, device="cuda"))     # float32 rows of a bf16 plan
    x = torch.zeros(s.rows, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mb.MlpBlkError):
        s.permute(x, x)


def test_positions_of_another_plan_stay_inside(mb):
    """pos of a larger batch handed to a smaller one's calls: entries beyond its rows
    count as none, and nothing outside the buffers is read or written."""
    import torch
    s = mb.MoeSort(4, 64, 3, 2, 16)
    pos = torch.tensor([[0, 1 << 20], [-7, 1], [s.rows, 2], [3, 2147483647]], dtype=torch.int32, device="cuda")
    count, seg = torch.tensor([5, 1 << 20, 0], dtype=torch.int32, device="cuda"), torch.tensor(
        [0, 16, 1 << 21, 1 << 22], dtype=torch.int32, device="cuda")
    whole = torch.full((s.rows * 64 + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    rows = whole[2048:2048 + s.rows * 64]
    x = torch.randn(4, 64, device="cuda").bfloat16()
    mb.mlpblk_moe_permute(s.desc, x, pos, count, seg, rows)
    got = rows.view(s.rows, 64)
    assert torch.equal(got[0], x[0]) and torch.equal(got[1], x[1]) and torch.equal(got[2], x[2]) and torch.equal(got[3], x[3])
    assert bool((whole[:2048] == 7).all()) and bool((whole[-2048:] == 7).all())
    y = torch.empty_like(x)
    mb.mlpblk_moe_unpermute(s.desc, rows, pos, None, None, y)
    assert torch.equal(y, x)


def test_rows_beyond_two_billion_elements(mb):
    """Sorted rows of more than 2^31 elements: both moves at their far end."""
    import torch
    T, d, E, k = 270000, 4096, 2, 2
    s = mb.MoeSort(T, d, E, k, 1)
    idx = torch.stack((torch.zeros(T), torch.ones(T)), 1).int().cuda()
    s.sort(idx)
    x = torch.arange(T, device="cuda", dtype=torch.float32)[:, None].remainder(251).expand(T, d).bfloat16().contiguous()
    rows = torch.zeros(s.rows, d, dtype=torch.bfloat16, device="cuda")
    assert rows.numel() > 1 << 31
    s.permute(x, rows)
    for t in (0, 1, T // 2, T - 1):
        assert torch.equal(rows[t], x[t]) and torch.equal(rows[T + t], x[t])
    y = torch.empty_like(x)
    s.permute_backward(rows, y)
    assert torch.equal(y, (2 * x.float()).bfloat16())
    dw = torch.empty(T, k, device="cuda")
    s.unpermute_backward(x, rows, None, y.new_zeros(s.rows, d), dw)
    ref = x[:, 0].float() ** 2 * d
    assert bool(((dw - ref[:, None]).abs() <= 2.0 ** -20 * ref[:, None]).all())


def test_plan_and_moves_of_two_billion_tokens(mb):
    """The largest plan that the descriptor takes with padding: its rows end within a warp's
    width of 2^31."""
    import torch
    T, pad = (1 << 31) - 5, 2
    s = mb.make_sort_desc(T, 1, 1, 1, pad)
    assert mb.mlpblk_moe_sort_rows(mb.make_sort_desc(T + 1, 1, 1, 1, pad)) == -1
    R = mb.mlpblk_moe_sort_rows(s)
    assert R == T + 1
    i32 = dict(dtype=torch.int32, device="cuda")
    idx = torch.zeros(T, **i32)
    idx[[3, T - 2]] = 1                                     # two ids that select nothing
    count, seg, pos, row_map = torch.zeros(1, **i32), torch.zeros(2, **i32), torch.zeros(T, **i32), torch.full((R + 64,), 7, **i32)
    mb.mlpblk_moe_sort(s, idx, count, seg, pos, row_map)
    assert count.item() == T - 2 and seg.tolist() == [0, T - 1]
    live = torch.ones(T, dtype=torch.bool, device="cuda")
    live[[3, T - 2]] = False
    entries = torch.nonzero(live)[:, 0].int()
    assert torch.equal(row_map[:T - 2], entries) and row_map[T - 2:R].tolist() == [-1] * 3 and bool((row_map[R:] == 7).all())
    del entries
    assert pos[3].item() == -1 and pos[T - 2].item() == -1
    assert torch.equal(row_map[pos[live].long()], torch.nonzero(live)[:, 0].int())
    del idx, row_map
    x = torch.arange(T, **i32).remainder_(251).to(torch.bfloat16)[:, None]
    rows = torch.full((R + 64, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    mb.mlpblk_moe_permute(s, x, pos, count, seg, rows)
    assert torch.equal(rows[:T - 2], x[live]) and rows[T - 2:, 0].tolist() == [0.0] + [7.0] * (R + 64 - T + 1)
    y = torch.full_like(x, 7.0)
    mb.mlpblk_moe_unpermute(s, rows, pos, None, None, y)
    x[~live] = 0.0
    assert torch.equal(y, x)
