"""Orthogonalised updates and Muon's step against the oracle (oracle.muon), GB300 only.

The tolerance is the documented 3e-3 of the Frobenius norm, plus bf16's half step (2^-8) for
the rounded result.  It comes from rounding each operand in float64 where the kernels round
it (fp16, 2^-11 a step of a value's binade): flat, steep and low-rank spectra of 64 x 64 to 768 x 768
gave 0.4e-3 to 2.3e-3; operands in bf16 would give 1e-2 and more, a step left out 1e-1.
"""

import numpy as np
import pytest

from oracle import muon

pytestmark = pytest.mark.gpu
NS, HALF = 3e-3, 2.0 ** -8


@pytest.fixture(scope="module")
def mb():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import mlp_block_backprop_gb300 as mb
    yield mb
    assert mb.mlpblk_last_error() == mb.MLPBLK_OK


def _exact(u, coefficients=(muon.COEFFICIENTS,) * 5, eps=1e-7):
    """The oracle's formula in float64 on the GPU."""
    import torch
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for a, b, c in coefficients:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _matrix(gen, r, c, kind, dtype):
    import torch
    dev = dict(device="cuda", generator=gen)
    u = torch.randn(r, c, **dev)
    if kind == "low":
        u = torch.randn(r, 3, **dev) @ torch.randn(3, c, **dev)
    elif kind == "mixed":
        k = min(16, r, c)
        u = 0.01 * u * (r ** 0.5 + c ** 0.5) / 2 + (torch.randn(r, k, **dev) / torch.arange(1, k + 1, device="cuda")) @ torch.randn(k, c, **dev)
    elif kind == "spike":
        u = 1e-6 * u
        u[r // 2, c // 3] = 1.0
    return u.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def _rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (33, 31), (63, 65), (64, 64), (100, 1000), (1000, 100), (127, 129), (128, 128),
          (129, 128), (255, 300), (333, 1000), (520, 333), (512, 2048), (2050, 640), (1, 5000), (5000, 3), (768, 776), (1300, 1290),
          (257, 9000), (9001, 260), (2048, 2048)]


@pytest.mark.parametrize("kind", ["flat", "low", "mixed"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(mb, shape, dtype, kind):
    import torch
    r, c = shape
    gen = torch.Generator(device="cuda").manual_seed(r * 7 + c)
    u = _matrix(gen, r, c, kind, dtype)
    before = u.clone()
    whole = torch.full((r * c + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = whole[256:256 + r * c].view(r, c)
    op = mb.Orthogonalizer(r, c, dtype=dtype)
    op._ws.fill_(0xFF)                         # scratch holds anything: here NaN
    op.orthogonalize(u, o)
    assert torch.equal(u, before)
    assert bool((whole[:256] == 7).all()) and bool((whole[-256:] == 7).all())
    assert _rel(o, _exact(u)) <= NS + HALF
    o2 = torch.empty_like(o)
    op.orthogonalize(u, o2)
    assert torch.equal(o, o2)


@pytest.mark.parametrize("shape", [(3, 96, 200), (5, 300, 130), (8, 1024, 512), (2, 1, 40), (40, 256, 256), (70, 64, 100)])
def test_batches(mb, shape):
    import torch
    b, r, c = shape
    gen = torch.Generator(device="cuda").manual_seed(b)
    u = torch.stack([_matrix(gen, r, c, ("flat", "mixed", "low")[i % 3], "f32") * 10.0 ** (i - 2) for i in range(b)])
    u[b // 2] = 0.0
    o = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
    mb.Orthogonalizer(r, c, batch=b, eps=1e-12).orthogonalize(u, o)
    for i in range(b):
        if i == b // 2:
            assert not o[i].any()
        elif bool(u[i].isfinite().all()):
            assert _rel(o[i], _exact(u[i], eps=1e-12)) <= NS + HALF
        else:                                       # from 10^38 on
            assert bool(o[i].isnan().all())


@pytest.mark.parametrize("steps", [1, 2, 3, 6])
@pytest.mark.parametrize("shape", [(150, 90), (90, 150), (700, 1400)])
def test_steps_of_their_own_coefficients(mb, shape, steps):
    import torch
    coef = [(2.0 - 0.1 * i, -1.5, 0.5 + 0.05 * i) for i in range(steps)]
    gen = torch.Generator(device="cuda").manual_seed(steps)
    u = _matrix(gen, *shape, "mixed", "f32")
    o = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    mb.Orthogonalizer(*shape, steps=steps, coefficients=coef).orthogonalize(u, o)
    assert _rel(o, _exact(u, coef)) <= NS + HALF


@pytest.mark.parametrize("steps", [2, 3, 4, 5, 6])
@pytest.mark.parametrize("shape", [(1, 1001, 4100), (1, 4500, 1024), (3, 700, 3001), (4, 2900, 650)])
def test_two_steps_with_one_product(mb, shape, steps):
    """Long sides of at least twice the short one, enough work: two steps share a product on X."""
    import torch
    b, r, c = shape
    gen = torch.Generator(device="cuda").manual_seed(steps)
    for kind in ("flat", "mixed", "low"):
        u = torch.stack([_matrix(gen, r, c, kind, "bf16") for _ in range(b)])
        o = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda")
        op = mb.Orthogonalizer(r, c, batch=b, steps=steps, dtype="bf16")
        op._ws.fill_(0xFF)
        with mb.KernelTrace(64) as trace:
            op.orthogonalize(u, o)
            torch.cuda.synchronize()
        names = [n for n, _ in trace.durations()]
        assert names.count("ns_join") == (steps - 1) // 2
        for i in range(b):
            assert _rel(o[i], _exact(u[i], (muon.COEFFICIENTS,) * steps)) <= NS + HALF


def test_zeros_without_eps(mb):
    import torch
    for shape in ((40, 70), (1300, 300)):
        u, o = torch.zeros(shape, device="cuda"), torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
        mb.Orthogonalizer(*shape, eps=0.0).orthogonalize(u, o)
        assert not o.any()


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-3, 1e10, 1e25, 1e36])
def test_size_of_u_does_not_matter(mb, scale):
    """Squares leave float32's range long before the values do."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    u = _matrix(gen, 200, 300, "flat", "f32") * scale
    o = torch.empty(200, 300, dtype=torch.bfloat16, device="cuda")
    mb.Orthogonalizer(200, 300, eps=0.0).orthogonalize(u, o)
    assert _rel(o, _exact(u, eps=0.0)) <= NS + HALF


def test_one_large_entry(mb):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(2)
    for shape in ((300, 500), (500, 300)):
        u = _matrix(gen, *shape, "spike", "f32")
        o = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        mb.Orthogonalizer(*shape).orthogonalize(u, o)
        assert _rel(o, _exact(u)) <= NS + HALF


def test_nan_stays_in_its_matrix(mb):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    u = torch.stack([_matrix(gen, 130, 70, "flat", "f32") for _ in range(3)])
    u[1, 4, 5] = float("nan")
    o = torch.empty(3, 130, 70, dtype=torch.bfloat16, device="cuda")
    mb.Orthogonalizer(130, 70, batch=3).orthogonalize(u, o)
    assert bool(o[1].isnan().all()) and _rel(o[0], _exact(u[0])) <= NS + HALF and _rel(o[2], _exact(u[2])) <= NS + HALF


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("case", [(1, 64, 64, "bf16"), (2, 130, 333, "f32"), (1, 515, 260, "bf16"), (3, 256, 1024, "bf16")])
def test_muon_steps(mb, case, nesterov):
    """Two steps; an update's error is NS times its norm, a weight has three roundings more."""
    import torch
    b, r, c, dtype = case
    gen = torch.Generator(device="cuda").manual_seed(r)
    w = torch.randn(b, r, c, device="cuda", generator=gen) * c ** -0.5
    m = torch.zeros_like(w)
    weight = torch.empty(b, r, c, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    gs = torch.tensor([0.5], device="cuda")
    op = mb.Orthogonalizer(r, c, batch=b, dtype=dtype)
    lr, beta, wd, scale = 0.02, 0.95, 0.1, 0.2 * max(r, c) ** 0.5
    for step in range(2):
        g = torch.stack([_matrix(gen, r, c, "mixed", "f32") for _ in range(b)])
        w0, m0 = w.double(), m.double()
        op.muon_step(w, g, m, lr, beta, wd, scale, nesterov, weight=weight, grad_scale=gs)
        for i in range(b):
            m1 = beta * m0[i] + 0.5 * g[i].double()
            assert _rel(m[i], m1) <= 4 * 2.0 ** -24 + 1e-8         # (beta as float32)
            x = _exact(0.5 * g[i].double() + beta * m1 if nesterov else m1)
            ref = w0[i] * (1 - lr * wd) - lr * scale * x
            tol = lr * scale * NS * float(x.norm()) + 4 * 2.0 ** -24 * float(ref.norm())
            assert float((w[i].double() - ref).norm()) <= tol
            assert torch.equal(weight[i], w[i].to(weight.dtype))


def test_two_streams_with_workspaces_of_their_own(mb):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(8)
    us = [_matrix(gen, 300, 400, "flat", "f32") for _ in range(2)]
    ops = [mb.Orthogonalizer(300, 400) for _ in range(2)]
    os_ = [torch.empty(300, 400, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            ops[i].orthogonalize(us[i], os_[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert _rel(os_[i], _exact(us[i])) <= NS + HALF


def test_capture_and_replay(mb):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    u = _matrix(gen, 256, 700, "flat", "f32")
    o = torch.empty(256, 700, dtype=torch.bfloat16, device="cuda")
    op = mb.Orthogonalizer(256, 700)
    op.orthogonalize(u, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.orthogonalize(u, o)
    u.copy_(_matrix(gen, 256, 700, "mixed", "f32"))
    g.replay()
    torch.cuda.synchronize()
    assert _rel(o, _exact(u)) <= NS + HALF


def test_offsets_beyond_32_bits(mb):
    """A batch of more than 2^32 elements: its first and last matrices."""
    import torch
    b, r, c = 70, 8192, 7500
    gen = torch.Generator(device="cuda").manual_seed(5)
    u = torch.empty(b, r, c, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    o = torch.zeros(b, r, c, dtype=torch.bfloat16, device="cuda")
    mb.Orthogonalizer(r, c, batch=b, steps=2, dtype="bf16").orthogonalize(u, o)
    for i in (0, b - 1):
        assert _rel(o[i], _exact(u[i], (muon.COEFFICIENTS,) * 2)) <= NS + HALF
