"""The router where float32 keys do not tell groups or experts apart, and gradients beside slots that select
nothing, against float64, GB300 only.  Ids are compared exactly; no tolerances but where stated."""

import numpy as np
import pytest

from oracle import route
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


def _select(l, k, score, bias, groups, top_groups):
    """oracle.route's ids for rows of finite logits and biases, all rows at once."""
    l = l.astype(np.float64)
    T, E = l.shape
    if score == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-l))
    else:
        e = np.exp(l - l.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True)
    key = s + bias.astype(np.float64)
    by = key.reshape(T, groups, E // groups)
    best = np.sort(by, axis=2)[:, :, -2:]
    marks = best.sum(axis=2)
    keep = np.argsort(-marks, axis=1, kind="stable")[:, :top_groups]
    kept = np.zeros((T, groups), dtype=bool)
    np.put_along_axis(kept, keep, True, axis=1)
    return np.argsort(-np.where(np.repeat(kept, E // groups, axis=1), key, -np.inf), axis=1, kind="stable")[:, :k].astype(np.int32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", [(256, 8, 4), (240, 10, 4), (48, 12, 5), (16, 8, 3)])
@pytest.mark.parametrize("size", [0.0, 1.0, 10.0, 100.0, 1e4])
def test_groups_whose_keys_cancel_in_their_marks(mb, shape, score, size):
    """A bias of +size on one expert of each group and -size on the others: marks near zero, whose keys'
    roundings are of +size's."""
    import torch
    E, groups, top_groups = shape
    T, k, per = 65536, 4, E // groups
    rng = np.random.default_rng(E)
    l = rng.normal(0, 0.1, (T, E)).astype(np.float32)
    bias = np.full((groups, per), -size, dtype=np.float32)
    bias[np.arange(groups), rng.integers(0, per, groups)] = size
    bias = bias.ravel()
    ids, w = torch.full((T, k), 77, dtype=torch.int32, device="cuda"), torch.full((T, k), 77.0, device="cuda")
    mb.MoeRouter(T, E, k, score, groups, top_groups, dtype="f32").route(torch.from_numpy(l).cuda(), ids, w, bias=torch.from_numpy(bias).cuda())
    ref = _select(l, k, score, bias, groups, top_groups)
    wrong = np.nonzero((ids.cpu().numpy() != ref).any(axis=1))[0]
    assert len(wrong) == 0, (len(wrong), wrong[:4], ids.cpu().numpy()[wrong[:4]], ref[wrong[:4]])
    some = slice(0, 40)
    np.testing.assert_array_equal(route.route(l[some], k, score, bias, groups, top_groups)[0], ref[some])


@pytest.mark.parametrize("shape", [(256, 8, 4), (240, 10, 4), (24, 12, 5)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_marks_beyond_the_range_of_float32(mb, shape, sign):
    """Biases of which two overflow when added: the marks order all the same."""
    import torch
    E, groups, top_groups = shape
    T, k = 300, 4
    rng = np.random.default_rng(groups)
    l = rng.normal(0, 1, (T, E)).astype(np.float32)
    bias = (sign * rng.uniform(1.8e38, 3.4e38, E)).astype(np.float32)
    ids, w = torch.full((T, k), 77, dtype=torch.int32, device="cuda"), torch.full((T, k), 77.0, device="cuda")
    mb.MoeRouter(T, E, k, "sigmoid", groups, top_groups, dtype="f32").route(torch.from_numpy(l).cuda(), ids, w, bias=torch.from_numpy(bias).cuda())
    ref, _ = route.route(l, k, "sigmoid", bias, groups, top_groups)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_beside_no_expert_have_no_part_in_the_gradient(mb, score, renorm, dtype):
    """d_routing_weights of slots without an expert (id -1, or an expert that is closed) may hold anything."""
    import torch
    T, E, k = 200, 40, 6
    rng = np.random.default_rng(1)
    l = rng.normal(0, 1, (T, E))
    l[rng.random((T, E)) < 0.9] = -np.inf                  # four open experts on average, six slots
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = torch.from_numpy(l.astype(np.float32)).to(dt).cuda()
    op = mb.MoeRouter(T, E, k, score, renorm=renorm, dtype=dtype)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    op.route(dev, ids, w)
    none = ids < 0
    assert bool(none.any()) and bool((~none).any())
    ids[:, 5] = torch.where(none[:, 5] & (dev[:, 7] == -float("inf")), 7, ids[:, 5])   # a closed expert's id
    dw = torch.from_numpy(rng.normal(0, 1, (T, k)).astype(np.float32)).cuda()
    want, got = torch.empty_like(dev), torch.empty_like(dev)
    op.route_backward(dev, ids, torch.where(none, 0.0, dw), want)
    assert bool(want.isfinite().all())
    for junk in (float("nan"), float("inf"), 3e38):
        op.route_backward(dev, ids, torch.where(none, junk, dw), got)
        assert torch.equal(got, want), junk
    ref = route.backward(to_np(dev), ids.cpu().numpy(), to_np(torch.where(none, 0.0, dw)), score, renorm)
    # (E + 12 roundings of 2^-24 of terms below 8, and half a step of the type)
    assert np.all(np.abs(to_np(want) - ref) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) + (E + 12) * 8 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [5, 40, 200])
def test_gradient_of_an_expert_named_twice(mb, E, score, renorm, dtype):
    """Ids of a caller's own, some experts in two slots and more: each slot adds its share."""
    import torch
    T, k = 70, 5
    rng = np.random.default_rng(E)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    dev = torch.from_numpy(rng.normal(0, 1, (T, E)).astype(np.float32)).to(dt).cuda()
    ids = rng.integers(0, min(E, 4), (T, k)).astype(np.int32)
    dw = rng.normal(0, 1, (T, k)).astype(np.float32)
    got = torch.full_like(dev, float("nan"))
    mb.MoeRouter(T, E, k, score, renorm=renorm, dtype=dtype).route_backward(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(dw).cuda(), got)
    ref = route.backward(to_np(dev), ids, dw, score, renorm)
    # terms: |dw| and their mean, at most 5 slots of them, over S >= s of the expert: below 64; E + 12 roundings of 2^-24, and
    # half a step of the type
    assert np.all(np.abs(to_np(got) - ref) <= (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) + (E + 12) * 64 * 2.0 ** -24)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,top_groups", [(16, 5), (64, 10), (9, 4)])
@pytest.mark.parametrize("size", [0.0, 10.0, 1e4])
def test_groups_of_one_expert(mb, E, top_groups, size, score):
    """A mark is half its only key; a common bias of `size` leaves the scores their last bits."""
    import torch
    T, k = 20000, 4
    rng = np.random.default_rng(E)
    l = rng.normal(0, 0.1, (T, E)).astype(np.float32)
    bias = np.full(E, size, dtype=np.float32)
    ids, w = torch.full((T, k), 77, dtype=torch.int32, device="cuda"), torch.full((T, k), 77.0, device="cuda")
    mb.MoeRouter(T, E, k, score, E, top_groups, dtype="f32").route(torch.from_numpy(l).cuda(), ids, w, bias=torch.from_numpy(bias).cuda())
    # (the k best of the best groups are the k best)
    ref = _select(l, k, score, bias, 1, 1)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)
