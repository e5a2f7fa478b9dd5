"""MXFP4 quantisation, reading back and products against the float64 oracle
(oracle.fp4), GB300 only.

Codes, scales and values read back are compared exactly: the scaling is by a power
of two and an element is rounded once.

Products: the operands' values are multiples of half their scale with at most 3
bits, so a block's 32 products add exactly; the K/32 scaled block sums are added in
float32.  Bound of an output: acc * sum|a||b| with acc = (K/32 + 2) * 2^-23 (one
float32 step, truncation included, an addition), plus half a step of the output
type (bf16 2^-8 relative to its value).  With all scales equal and small integers
every partial sum is a multiple of 1/4 below 2^22, so those products are exact.
"""

import numpy as np
import pytest

import fp4_shapes
from oracle import fp4, sort
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


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _dev(a, dtype):
    import torch
    return torch.from_numpy(np.array(a, dtype=np.float32)).cuda().to(_dt(dtype))


def _draw(rng, shape, dtype):
    """Normal values with blocks of very different sizes, some of them zero."""
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-20, 20, size=(shape[0], 1)))
    v[rng.random(shape) < 0.05] = 0.0
    if shape[0] > 3:
        v[2] = 0.0
    t = _dev(v, dtype)
    return t, to_np(t)


def _bytes(t):
    return t.cpu().numpy()


# ------------------------------------------------------- quantise and read back

SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (8, 4096), (31, 256), (127, 257), (128, 128), (129, 1000), (300, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_rows(mb, shape, dtype):
    import torch
    x, v = _draw(np.random.default_rng(sum(shape)), shape, dtype)
    q = mb.Fp4Matrix(*shape)
    q.codes.fill_(0xAA)
    q.scales.fill_(0xAA)
    q.quantize(x)
    codes, scales = fp4.quantize(v)
    packed, tiled = fp4.pack(codes, scales)
    np.testing.assert_array_equal(_bytes(q.scales), tiled)
    np.testing.assert_array_equal(_bytes(q.codes), packed)
    for out in ("bf16", "f32"):
        y = torch.full(shape, float("nan"), dtype=_dt(out), device="cuda")
        q.dequantize(y)
        np.testing.assert_array_equal(to_np(y), fp4.values(codes, scales, shape[1]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_transposed(mb, shape, dtype):
    x, v = _draw(np.random.default_rng(sum(shape) + 1), shape[::-1], dtype)
    q = mb.Fp4Matrix(*shape)
    q.codes.fill_(0xAA)
    q.scales.fill_(0xAA)
    q.quantize(x, transposed=True)
    packed, tiled = fp4.pack(*fp4.quantize(v.T))
    np.testing.assert_array_equal(_bytes(q.scales), tiled)
    np.testing.assert_array_equal(_bytes(q.codes), packed)


@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_relu2_and_special_values(mb, transposed):
    rng = np.random.default_rng(3)
    v = rng.standard_normal((70, 100))
    v[4, 5], v[40, 70], v[69, 99], v[10, 10] = np.inf, np.nan, -np.inf, 3e38
    v[20, :] = 1e-39                                        # float32 subnormals
    x = _dev(v, "f32")
    w = to_np(x).T if transposed else to_np(x)
    for act in ("none", "relu2"):
        a = w
        if act == "relu2":
            a = np.where(w < 0, 0.0, w).astype(np.float32)
            with np.errstate(over="ignore"):
                a = (a * a).astype(np.float64)             # float32 squares: the largest becomes infinite
        q = mb.Fp4Matrix(*w.shape)
        q.quantize(x, transposed=transposed, act=act)
        packed, tiled = fp4.pack(*fp4.quantize(a))
        np.testing.assert_array_equal(_bytes(q.scales), tiled)
        np.testing.assert_array_equal(_bytes(q.codes) & 0x77, packed & 0x77)
        import torch
        y = torch.empty(w.shape, dtype=torch.float32, device="cuda")
        q.dequantize(y)
        np.testing.assert_array_equal(to_np(y), fp4.rounded(a))


@pytest.mark.parametrize("act", ["none", "relu2"])
@pytest.mark.parametrize("shape", [(9, 33), (40, 31), (130, 7), (33, 258), (64, 289), (70, 1031), (17, 2049), (5, 1028)])
def test_rows_that_begin_anywhere(mb, shape, act):
    """bf16 rows of every alignment, with NaN right behind the matrix: what is not the
    row's reaches no code; values read back stop at the matrix's end."""
    import torch
    rows, cols = shape
    buf = torch.full((rows * cols + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, v = _draw(np.random.default_rng(cols), shape, "bf16")
    v[rows // 2, cols // 2:] = np.inf
    v[rows - 1, 0] = np.nan
    buf[:rows * cols] = torch.from_numpy(v.astype(np.float32)).cuda().to(torch.bfloat16).reshape(-1)
    a = v if act == "none" else np.where(v < 0, 0.0, v * v)
    q = mb.Fp4Matrix(rows, cols)
    q.codes.fill_(0xAA)
    q.scales.fill_(0xAA)
    q.quantize(buf[:rows * cols].view(rows, cols), act=act)
    packed, tiled = fp4.pack(*fp4.quantize(a))
    np.testing.assert_array_equal(_bytes(q.scales), tiled)
    mask = 0xFF if act == "none" else 0x77
    np.testing.assert_array_equal(_bytes(q.codes) & mask, packed & mask)
    for dt in ("bf16", "f32"):
        y = torch.full((rows * cols + 64,), 7.0, dtype=_dt(dt), device="cuda")
        q.dequantize(y[:rows * cols].view(rows, cols))
        np.testing.assert_array_equal(to_np(y[:rows * cols]).reshape(shape), fp4.rounded(a))
        assert (y[rows * cols:] == 7.0).all()


@pytest.mark.parametrize("cols", [32, 31, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_read_back_every_code_and_scale(mb, dtype, cols):
    import torch
    q = mb.Fp4Matrix(256, cols)
    r = np.arange(256)
    scales = np.zeros((2, 2, 512), dtype=np.uint8)          # row r has the scale byte r in each of its blocks
    for b in range(4):
        scales[r // 128, 0, r % 32 * 16 + r % 128 // 32 * 4 + b] = r
    nib = np.arange(cols + 32) % 16
    q.scales.copy_(torch.from_numpy(scales.reshape(-1)).cuda())
    ld = (cols + 31) // 32 * 16
    row = (nib[0:2 * ld:2] | nib[1:2 * ld:2] << 4).astype(np.uint8)
    q.codes.copy_(torch.from_numpy(np.tile(row, (256, 1))).cuda().reshape(q.codes.shape))
    y = torch.empty(256, cols, dtype=_dt(dtype), device="cuda")
    q.dequantize(y)
    size = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    ref = (np.where(nib[:cols] < 8, 1.0, -1.0) * size[nib[:cols] % 8])[None, :] * np.exp2(r - 127.0)[:, None]
    ref[255] = np.nan
    with np.errstate(over="ignore"):
        ref = ref.astype(np.float32)                        # beyond 2^128: infinite
    np.testing.assert_array_equal(to_np(y), ref)
    np.testing.assert_array_equal(np.signbit(to_np(y)[:255]), np.signbit(ref[:255]))


def test_quantize_batch(mb):
    import torch
    x, v = _draw(np.random.default_rng(4), (3 * 130, 72), "bf16")
    q = mb.Fp4Matrix(130, 72, batch=3)
    q.quantize(x)
    packs = [fp4.pack(*fp4.quantize(v[130 * i:130 * i + 130])) for i in range(3)]
    np.testing.assert_array_equal(_bytes(q.codes), np.concatenate([p[0] for p in packs]))
    np.testing.assert_array_equal(_bytes(q.scales), np.concatenate([p[1] for p in packs]))
    y = torch.empty(3, 130, 72, dtype=torch.float32, device="cuda")
    q.dequantize(y)
    np.testing.assert_array_equal(to_np(y), np.stack([fp4.rounded(v[130 * i:130 * i + 130]) for i in range(3)]))
    qt = mb.Fp4Matrix(72, 130, batch=3)
    qt.quantize(x, transposed=True)
    packs = [fp4.pack(*fp4.quantize(v[130 * i:130 * i + 130].T)) for i in range(3)]
    np.testing.assert_array_equal(_bytes(qt.codes), np.concatenate([p[0] for p in packs]))
    np.testing.assert_array_equal(_bytes(qt.scales), np.concatenate([p[1] for p in packs]))


def _routed(mb, T, width, E, k, pad, seed, dead=()):
    import torch
    rng = np.random.default_rng(seed)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    for e in dead:
        idx[idx == e] = (e + 1) % E
    if T > 2 and k > 1:
        idx[1, 0] = -1
        idx[2, :] = idx[2, 0]                               # an expert named k times
    s = mb.MoeSort(T, width, E, k, pad)
    s.sort(torch.from_numpy(idx).cuda())
    return s, sort.plan(idx, E, pad)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", [(45, 90, 5, 2, 128), (6, 301, 40, 2, 256), (37, 1032, 9, 3, 128)])
def test_quantize_through_a_sort(mb, shape, transposed, gather):
    import torch
    T, d, E, k, pad = shape
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, pad, 5)
    R = s.rows
    x, v = _draw(np.random.default_rng(6), (T if gather else R, d), "bf16")
    live = row_map >= 0
    src = np.where(live[:, None], v[np.maximum(row_map, 0) // k] if gather else v, 0.0)
    if not gather:                                          # what no entry owns is not read
        x[torch.from_numpy(~live).cuda()] = float("nan")
    shape = (d, R) if transposed else (R, d)
    q = mb.Fp4Matrix(*shape)
    q.quantize(x, sort=s, gather=gather, transposed=transposed)
    packed, tiled = fp4.pack(*fp4.quantize(src.T if transposed else src))
    np.testing.assert_array_equal(_bytes(q.scales), tiled)
    np.testing.assert_array_equal(_bytes(q.codes), packed)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("d", [64, 90, 101])
def test_rows_mapped_beyond_the_source_are_zeros(mb, d, transposed, dtype):
    """A gathering map of a larger batch: entries at or behind the source's last row come
    out as zero blocks, and what lies around the source (NaN here) reaches no code."""
    import torch
    T, R, div = 21, 300, 3
    rng = np.random.default_rng(d)
    row_map = rng.integers(-3, 3 * T * div, R).astype(np.int32)
    row_map[:4] = [T * div - 1, T * div, 2 ** 31 - 1, -2 ** 31]
    whole = torch.full((2 * 64 * d + T * d,), float("nan"), dtype=_dt(dtype), device="cuda")
    x, v = _draw(rng, (T, d), dtype)
    whole[64 * d:64 * d + T * d] = x.reshape(-1)
    at = np.where(row_map >= 0, row_map // div, T)
    src = np.where((at < T)[:, None], v[np.minimum(at, T - 1)], 0.0)
    packed, tiled = fp4.pack(*fp4.quantize(src.T if transposed else src))
    shape = (d, R) if transposed else (R, d)
    rm = torch.from_numpy(row_map).cuda()
    q = mb.Fp4Matrix(*shape)
    # the rows stated, and (0) those that the tensor has
    for rows, xs in ((T, whole[64 * d:]), (0, whole[64 * d:64 * d + T * d])):
        q.codes.fill_(0xAA)
        q.scales.fill_(0xAA)
        mb.mlpblk_fp4_quantize(mb.make_fp4_desc(*shape, dtype=dtype, transposed=transposed, source_rows=rows), xs,
                               q.codes, q.scales, row_map=rm, map_div=div)
        np.testing.assert_array_equal(_bytes(q.scales), tiled)
        np.testing.assert_array_equal(_bytes(q.codes), packed)
    with pytest.raises(mb.MlpBlkError):                     # fewer rows than stated
        mb.mlpblk_fp4_quantize(mb.make_fp4_desc(*shape, dtype=dtype, transposed=transposed, source_rows=T + 1),
                               x, q.codes, q.scales, row_map=rm, map_div=div)


# ---------------------------------------------------------------------- products

def _check(got, a, b, out, k, base=None):
    ref, mag = fp4.product(a, b)
    if base is not None:
        ref, mag = ref + base, mag + np.abs(base)
    tol = (-(-k // 32) + 2 + (base is not None)) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if out == "bf16" else 0.0)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4])


def _quantized(mb, rng, rows, cols, batch=1, wide=True):
    import torch
    v = rng.standard_normal((batch * rows, cols))
    if wide:
        v *= np.exp2(rng.integers(-6, 6, size=(batch * rows, 1)))
    x = torch.from_numpy(v.astype(np.float32)).cuda()
    q = mb.Fp4Matrix(rows, cols, batch=batch)
    q.quantize(x)
    vals = np.stack([fp4.rounded(to_np(x)[i * rows:(i + 1) * rows]) for i in range(batch)])
    return q, vals if batch > 1 else vals[0]


@pytest.mark.parametrize("shape", [(1, 128, 256), (32, 128, 64), (128, 128, 1024), (256, 512, 512), (2560, 2048, 1024)])
def test_product_exact(mb, shape):
    """Codes of every value with scale 1, each row its own pattern: sums are exact,
    and a wrong lane, column, K order or scale would show."""
    import torch
    m, n, k = shape
    rng = np.random.default_rng(k)
    a = rng.choice(np.concatenate([fp4.VALUES, -fp4.VALUES]), size=(m, k))
    b = rng.choice(np.concatenate([fp4.VALUES, -fp4.VALUES]), size=(n, k))
    a[:, ::32], b[:, ::32] = 6.0, -6.0                       # every block's scale is 1
    qa, qb = mb.Fp4Matrix(m, k), mb.Fp4Matrix(n, k)
    qa.quantize(torch.from_numpy(a.astype(np.float32)).cuda())
    qb.quantize(torch.from_numpy(b.astype(np.float32)).cuda())
    c = torch.full((m, n), float("nan"), device="cuda")
    qa.matmul(qb, c)
    np.testing.assert_array_equal(to_np(c), a @ b.T)


@pytest.mark.parametrize("m,n", [(1, 256), (32, 256), (128, 256), (2560, 2048)])
def test_product_scales(mb, m, n):
    """One non-zero element a row, scales that differ by row and block: each output is
    one exact product, so every scale must reach its own row and block of K."""
    import torch
    k = 1024
    rng = np.random.default_rng(m)
    a, b = np.zeros((m, k)), np.exp2(rng.integers(-8, 8, size=(n, k // 32))).repeat(32, axis=1)
    a[np.arange(m), rng.integers(0, k, m)] = np.exp2(rng.integers(-8, 8, m))
    qa, qb = mb.Fp4Matrix(m, k), mb.Fp4Matrix(n, k)
    qa.quantize(torch.from_numpy(a.astype(np.float32)).cuda())
    qb.quantize(torch.from_numpy(b.astype(np.float32)).cuda())
    c = torch.full((m, n), float("nan"), device="cuda")
    qa.matmul(qb, c)
    np.testing.assert_array_equal(to_np(c), a @ b.T)


PRODUCTS = [
    (1, 1, 1), (1, 130, 32), (2, 64, 100), (8, 1000, 2049), (31, 257, 4096), (33, 129, 255), (40, 4096, 300),
    (128, 256, 256), (129, 127, 512), (333, 1000, 1031), (257, 384, 8200), (1, 300, 16384), (1000, 70, 640),
    (512, 1024, 768), (1025, 2050, 1000), (2048, 2048, 512), (2305, 1536, 288), (4, 16384, 4096),
    (2100, 2056, 320), (2100, 2052, 320),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PRODUCTS)
def test_product(mb, shape, out):
    import torch
    m, n, k = shape
    rng = np.random.default_rng(m + n + k)
    qa, a = _quantized(mb, rng, m, k)
    qb, b = _quantized(mb, rng, n, k)
    c = torch.full((m, n), float("nan"), dtype=_dt(out), device="cuda")
    qa.matmul(qb, c)
    _check(to_np(c), a, b, out, k)


@pytest.mark.parametrize("shape", [(1, 130, 64), (33, 129, 300), (200, 256, 2048), (1030, 1100, 520), (2048, 2304, 300)])
def test_product_accumulates(mb, shape):
    import torch
    m, n, k = shape
    rng = np.random.default_rng(m)
    qa, a = _quantized(mb, rng, m, k)
    qb, b = _quantized(mb, rng, n, k)
    c = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda()
    base = to_np(c)
    qa.matmul(qb, c, accumulate=True)
    _check(to_np(c), a, b, "f32", k, base)


def test_product_leaves_the_neighbours_alone(mb):
    """C in the middle of a larger buffer: nothing before or behind it is touched."""
    import torch
    rng = np.random.default_rng(8)
    for m, n, k in ((5, 100, 64), (300, 333, 96), (700, 1000, 64)):
        for out in ("bf16", "f32"):
            qa, a = _quantized(mb, rng, m, k)
            qb, b = _quantized(mb, rng, n, k)
            whole = torch.full((m * n + 2048,), 7.0, dtype=_dt(out), device="cuda")
            c = whole[1024:1024 + m * n]
            mb.mlpblk_fp4_matmul(mb.make_fp4_matmul_desc(m, n, k, out), qa.codes, qa.scales, qb.codes, qb.scales, c)
            _check(to_np(c).reshape(m, n), a, b, out, k)
            assert bool((whole[:1024] == 7.0).all()) and bool((whole[1024 + m * n:] == 7.0).all())


@pytest.mark.parametrize("m", [3, 200, 600])
def test_product_nan_rows_stay_in_their_row(mb, m):
    import torch
    n, k = 300, 512
    rng = np.random.default_rng(9)
    va, vb = rng.standard_normal((m, k)), rng.standard_normal((n, k))
    va[1, 40], vb[70, 300] = np.nan, np.inf
    qa, qb = mb.Fp4Matrix(m, k), mb.Fp4Matrix(n, k)
    qa.quantize(_dev(va, "f32"))
    qb.quantize(_dev(vb, "f32"))
    c = torch.zeros(m, n, device="cuda")
    qa.matmul(qb, c)
    got = to_np(c)
    nan = np.zeros((m, n), dtype=bool)
    nan[1], nan[:, 70] = True, True
    assert np.array_equal(np.isnan(got), nan)
    a, b = fp4.rounded(_np32(va)), fp4.rounded(_np32(vb))
    keep_r, keep_c = np.arange(m) != 1, np.arange(n) != 70
    _check(got[keep_r][:, keep_c], a[keep_r], b[keep_c], "f32", k)


def _np32(v):
    return np.asarray(v, dtype=np.float32).astype(np.float64)


# (T, d, n, E, k, pad)
GROUPED = [(1, 64, 130, 3, 2, 128), (8, 256, 512, 8, 2, 128), (40, 300, 200, 5, 2, 128), (300, 96, 333, 7, 3, 256),
           (700, 520, 640, 4, 2, 128), (2000, 256, 1024, 3, 2, 256), (513, 128, 64, 200, 4, 128),
           (3000, 200, 1000, 5, 2, 128), (3000, 136, 1001, 5, 2, 128)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("case", GROUPED)
def test_grouped_product(mb, case, out):
    import torch
    T, d, n, E, k, pad = case
    rng = np.random.default_rng(T + n)
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, pad, T, dead=(1,))
    x, v = _draw(rng, (T, d), "bf16")
    qx = mb.Fp4Matrix(s.rows, d)
    qx.quantize(x, sort=s, gather=True)
    qw, w = _quantized(mb, rng, n, d, batch=E)
    c = torch.full((s.rows, n), 7.0, dtype=_dt(out), device="cuda")
    qx.matmul_grouped(qw, s, c)
    got = to_np(c)
    a = fp4.rounded(np.where((row_map >= 0)[:, None], v[np.maximum(row_map, 0) // k], 0.0))
    for e in range(E):
        r = slice(seg[e], seg[e] + count[e])
        if count[e]:
            _check(got[r], a[r], w[e], out, d)
        pad_rows = got[seg[e] + count[e]:seg[e + 1]]
        assert np.all((pad_rows == 0.0) | (pad_rows == 7.0))
    assert np.all(got[seg[E]:] == 7.0)
    if out == "f32":
        base = torch.from_numpy(rng.standard_normal((s.rows, n)).astype(np.float32)).cuda()
        b0 = to_np(base)
        qx.matmul_grouped(qw, s, base, accumulate=True)
        got = to_np(base)
        for e in range(E):
            r = slice(seg[e], seg[e] + count[e])
            if count[e]:
                _check(got[r], a[r], w[e], out, d, b0[r])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", [(1, 64, 130, 3, 2), (40, 300, 200, 5, 2), (300, 96, 333, 7, 3), (2000, 256, 520, 4, 2),
                                  (1000, 1024, 1200, 6, 2), (1000, 1023, 1200, 6, 2)])
def test_grouped_wgrad(mb, case, accumulate):
    import torch
    T, d, n, E, k = case
    rng = np.random.default_rng(T + n + 1)
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, 256, T, dead=(0,))
    live = (row_map >= 0)[:, None]
    x, v = _draw(rng, (T, d), "bf16")
    dy, g = _draw(rng, (s.rows, n), "bf16")
    qx, qg = mb.Fp4Matrix(d, s.rows), mb.Fp4Matrix(n, s.rows)
    qx.quantize(x, sort=s, gather=True, transposed=True)
    qg.quantize(dy, sort=s, transposed=True)
    a = fp4.rounded(np.where(live, g, 0.0).T)
    b = fp4.rounded(np.where(live, v[np.maximum(row_map, 0) // k], 0.0).T)
    c = torch.from_numpy(rng.standard_normal((E, n, d)).astype(np.float32)).cuda()
    base = to_np(c)
    qg.wgrad_grouped(qx, s, c, accumulate=accumulate)
    got = to_np(c)
    for e in range(E):
        r = slice(seg[e], seg[e + 1])
        _check(got[e], a[:, r], b[:, r], "f32", seg[e + 1] - seg[e], base[e] if accumulate else None)
    assert count[0] == 0 and np.array_equal(got[0], base[0] if accumulate else np.zeros((n, d)))


def test_experts_together(mb):
    """The routed ReLU^2 experts at 4 bits as a program runs them: sort, quantise the
    gathered tokens, up product, ReLU^2 and quantise, down product, weighted sum with
    the residual; each stage against the oracle on the stage's own input."""
    import torch
    T, d, F, E, k, pad = 150, 160, 288, 5, 2, 128
    rng = np.random.default_rng(10)
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, pad, 11)
    live = (row_map >= 0)[:, None]
    x = _dev(rng.standard_normal((T, d)), "bf16")
    v = to_np(x)
    w1, b1 = _quantized(mb, rng, F, d, batch=E, wide=False)
    w2, b2 = _quantized(mb, rng, d, F, batch=E, wide=False)
    p = torch.rand(T, k, device="cuda")
    qx, qh = mb.Fp4Matrix(s.rows, d), mb.Fp4Matrix(s.rows, F)
    h = torch.full((s.rows, F), float("nan"), dtype=torch.bfloat16, device="cuda")
    o = torch.full((s.rows, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    qx.quantize(x, sort=s, gather=True)
    qx.matmul_grouped(w1, s, h)
    qh.quantize(h, sort=s, act="relu2")
    qh.matmul_grouped(w2, s, o)
    s.unpermute(o, y, weights=p, residual=x)
    a = fp4.rounded(np.where(live, v[np.maximum(row_map, 0) // k], 0.0))
    hq = np.where(live, to_np(h), 0.0)
    aq = fp4.rounded(np.square(np.maximum(hq, 0.0)))
    for e in range(E):
        r = slice(seg[e], seg[e] + count[e])
        _check(to_np(h)[r], a[r], b1[e], "bf16", d)
        _check(to_np(o)[r], aq[r], b2[e], "bf16", F)
    ref, mag = sort.unpermute(np.where(live, to_np(o), 0.0), pos, to_np(p), v)
    assert np.all(np.abs(to_np(y) - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 2) * 2.0 ** -24 * mag)


def test_linear_gradients_against_differences(mb):
    """dx and dW of y = Q(x) Q(W)^T as the three products give them, for a loss that is
    linear in y, against differences of the exact product: with x, W and dy already
    MXFP4 values along both axes (small integers, scale 1), quantisation changes
    nothing and the gradients are exact."""
    import torch
    m, n, k = 64, 96, 160
    rng = np.random.default_rng(12)
    draw = lambda r, c: rng.choice([-6.0, -3.0, -1.0, 0.5, 2.0, 4.0, 6.0], size=(r, c))
    x, w, dy = draw(m, k), draw(n, k), draw(m, n)
    for t in (x, w, dy):
        t[::32, :], t[:, ::32] = 6.0, 6.0
    q = lambda a, tr=False: _q(mb, a, tr)
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    q(dy).matmul(q(w, True), dx)
    q(dy, True).matmul(q(x, True), dw)
    loss = lambda x, w: float(np.sum((x @ w.T) * dy))
    for i, j in ((0, 0), (63, 159), (17, 31)):
        e = np.zeros_like(x)
        e[i, j] = 1.0
        assert to_np(dx)[i, j] == (loss(x + e, w) - loss(x - e, w)) / 2
    for i, j in ((0, 0), (95, 159), (33, 64)):
        e = np.zeros_like(w)
        e[i, j] = 1.0
        assert to_np(dw)[i, j] == (loss(x, w + e) - loss(x, w - e)) / 2


def _q(mb, a, transposed):
    rows, cols = a.shape[::-1] if transposed else a.shape
    m = mb.Fp4Matrix(rows, cols)
    m.quantize(_dev(a, "f32"), transposed=transposed)
    return m


def test_streams_and_graph(mb):
    """Two streams at once with their own buffers, then a captured graph replayed on
    new inputs."""
    import torch
    m, n, k = 64, 512, 1024
    rng = np.random.default_rng(13)
    qw, w = _quantized(mb, rng, n, k)
    xs = [torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).cuda() for _ in range(2)]
    qs = [mb.Fp4Matrix(m, k) for _ in range(2)]
    cs = [torch.empty(m, n, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                qs[i].quantize(xs[i])
                qs[i].matmul(qw, cs[i])
    torch.cuda.synchronize()
    for i in range(2):
        _check(to_np(cs[i]), fp4.rounded(to_np(xs[i])), w, "f32", k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs[0].quantize(xs[0])
        qs[0].matmul(qw, cs[0])
    for _ in range(2):
        xs[0].normal_()
        cs[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        _check(to_np(cs[0]), fp4.rounded(to_np(xs[0])), w, "f32", k)


def test_binding_checks(mb):
    import torch
    q = mb.Fp4Matrix(8, 64)
    x = torch.zeros(8, 128, device="cuda")
    for bad in (x[:, ::2], x[:, :64], torch.zeros(8, 63, device="cuda"), torch.zeros(8, 64)):
        with pytest.raises(mb.MlpBlkError):
            q.quantize(bad)
    with pytest.raises(mb.MlpBlkError):
        q.quantize(torch.zeros(8, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(mb.MlpBlkError):
        q.matmul(mb.Fp4Matrix(8, 96), torch.zeros(8, 8, device="cuda"))
    with pytest.raises(mb.MlpBlkError):
        q.matmul(q, torch.zeros(8, 7, device="cuda"))
    with pytest.raises(mb.MlpBlkError):
        q.matmul(q, torch.zeros(8, 8, device="cuda", dtype=torch.bfloat16), accumulate=True)


def test_wgrad_of_no_rows(mb):
    import torch
    s = mb.MoeSort(0, 64, 4, 2, 256)
    s.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert s.rows == 0 and not s.count.any() and not s.seg.any()
    a, b = mb.Fp4Matrix(32, 0), mb.Fp4Matrix(64, 0)
    c = torch.full((4, 32, 64), 3.0, device="cuda")
    a.wgrad_grouped(b, s, c, accumulate=True)
    assert bool((c == 3.0).all())
    a.wgrad_grouped(b, s, c)
    assert not c.any()


def test_no_row_chosen(mb):
    """Every id invalid: no tile at all, C as it was; weight gradients zero."""
    import torch
    for T, E in ((5, 4), (3000, 6)):
        s = mb.MoeSort(T, 64, E, 2, 256)
        s.sort(torch.full((T, 2), -1, dtype=torch.int32, device="cuda"))
        x = torch.randn(T, 64, device="cuda")
        q, qt, w = mb.Fp4Matrix(s.rows, 64), mb.Fp4Matrix(64, s.rows), mb.Fp4Matrix(96, 64, batch=E)
        q.quantize(x, sort=s, gather=True)
        qt.quantize(x, sort=s, gather=True, transposed=True)
        w.quantize(torch.randn(E * 96, 64, device="cuda"))
        c = torch.full((s.rows, 96), 5.0, device="cuda")
        q.matmul_grouped(w, s, c)
        assert bool((c == 5.0).all())
        dw = torch.full((E, 64, 64), 5.0, device="cuda")
        qt.wgrad_grouped(qt, s, dw)
        assert not dw.any()


def test_repeats_are_bitwise_equal(mb):
    import torch
    rng = np.random.default_rng(14)
    for m, n, k in ((3, 4096, 8192), (200, 600, 4000), (2300, 2304, 1000)):
        qa, _ = _quantized(mb, rng, m, k)
        qb, _ = _quantized(mb, rng, n, k)
        outs = []
        for _ in range(3):
            c = torch.full((m, n), 1.0, device="cuda")
            qa.matmul(qb, c, accumulate=True)
            outs.append(c)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_matrices_beyond_two_billion_elements(mb):
    """A source and a C of more than 2^31 elements, at their far ends."""
    import torch
    rows, cols = 70000, 32768
    x = torch.randn(256, cols, device="cuda").bfloat16().repeat(rows // 256 + 1, 1)[:rows].contiguous()
    assert x.numel() > 1 << 31
    tail = x[rows - 300:].contiguous()
    for tr in (False, True):
        if tr:
            x, tail = x.view(cols, rows), x.view(cols, rows)[:, rows - 300:].contiguous()
        q, qs = mb.Fp4Matrix(rows, cols), mb.Fp4Matrix(300, cols)
        q.quantize(x, transposed=tr)
        qs.quantize(tail, transposed=tr)
        assert torch.equal(q.codes.view(rows, -1)[rows - 300:], qs.codes.view(300, -1))
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    q.dequantize(y)
    ys = torch.empty(300, cols, dtype=torch.bfloat16, device="cuda")
    qs.dequantize(ys)
    assert torch.equal(y[rows - 300:], ys)
    del x, y, q, qs, ys, tail
    for m, n in ((46400, 46400), (30, 75_000_000)):
        a, b = torch.randn(m, 64, device="cuda"), torch.randn(n, 64, device="cuda")
        qa, qb = mb.Fp4Matrix(m, 64), mb.Fp4Matrix(n, 64)
        qa.quantize(a)
        qb.quantize(b)
        c = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        assert c.numel() > 1 << 31
        qa.matmul(qb, c)
        i, j = slice(m - 20, m), slice(n - 200, n)
        _check(to_np(c[i, j]), fp4.rounded(to_np(a[i])), fp4.rounded(to_np(b[j])), "bf16", 64)
        _check(to_np(c[:20, j]), fp4.rounded(to_np(a[:20])), fp4.rounded(to_np(b[j])), "bf16", 64)


def test_without_the_native_calls(mb, monkeypatch):
    """The classes through ctypes, as on a machine without Python's headers."""
    import types
    names = ("moe_sort", "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
             "fp4_quantize", "fp4_dequantize", "fp4_matmul", "fp4_matmul_grouped", "fp4_wgrad_grouped")
    monkeypatch.setattr(mb, "_calls", types.SimpleNamespace(**{n: mb._Calls._ctypes("mlpblk_" + n) for n in names}))
    test_experts_together(mb)
    test_grouped_wgrad(mb, (40, 300, 200, 5, 2), True)
    test_quantize_rows(mb, (5, 33), "f32")


def test_buffers_that_only_touch(mb):
    """Every buffer of a pass cut from one allocation, each directly behind the one before:
    nothing is refused, nothing is written beyond its own bytes."""
    import torch
    T, d, n, E, k, pad = 40, 96, 72, 4, 2, 256
    rng = np.random.default_rng(21)
    s0 = mb.MoeSort(T, d, E, k, pad)
    R = s0.rows
    whole = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    at = [0]

    def cut(shape, dtype):
        size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        assert size % 16 == 0
        at[0] += size
        return whole[at[0] - size:at[0]].view(dtype).view(shape)

    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    idx, count, seg4 = cut((T, k), i32), cut((E,), i32), cut((8,), i32)
    seg, pos, row_map = seg4[:E + 1], cut((T, k), i32), cut((R,), i32)
    x, rows, w, y = cut((T, d), f32), cut((R, d), f32), cut((T, k), f32), cut((T, d), f32)
    dr, dw, dx = cut((R, d), f32), cut((T, k), f32), cut((T, d), f32)
    fp4_of = lambda r, c, b=1: (cut((r * b * -(-c // 32) * 16,), u8), cut((-(-r // 128) * -(-c // 256) * 1024 * b,), u8))
    a, bt, at_, = fp4_of(R, d), fp4_of(n, d, E), fp4_of(d, R)
    c, back, g = cut((R, n), f32), cut((R, d), f32), cut((E, d, d), f32)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    idx.copy_(torch.from_numpy(ids))
    x.normal_()
    w.fill_(0.5)
    wn = torch.randn(E * n, d, device="cuda")
    desc = mb.make_sort_desc(T, d, E, k, pad, "f32")
    mb.mlpblk_moe_sort(desc, idx, count, seg, pos, row_map)
    mb.mlpblk_moe_permute(desc, x, pos, count, seg, rows)
    mb.mlpblk_moe_unpermute(desc, rows, pos, w, x, y)
    mb.mlpblk_moe_unpermute_backward(desc, y, rows, pos, count, seg, w, dr, dw)
    mb.mlpblk_moe_permute_backward(desc, rows, pos, dx)
    mb.mlpblk_fp4_quantize(mb.make_fp4_desc(R, d, dtype="f32", source_rows=T), x, *a, row_map=row_map, map_div=k)
    mb.mlpblk_fp4_quantize(mb.make_fp4_desc(n, d, E, dtype="f32"), wn, *bt)
    mb.mlpblk_fp4_quantize(mb.make_fp4_desc(d, R, dtype="f32", transposed=True, source_rows=T), x, *at_, row_map=row_map, map_div=k)
    mb.mlpblk_fp4_matmul_grouped(mb.make_fp4_matmul_desc(R, n, d, "f32", experts=E, pad=pad), *a, *bt, count, seg, c)
    mb.mlpblk_fp4_dequantize(mb.make_fp4_desc(R, d, dtype="f32"), *a, back)
    mb.mlpblk_fp4_wgrad_grouped(mb.make_fp4_matmul_desc(d, d, R, "f32", experts=E, pad=pad), *at_, *at_, seg, g)
    assert not whole[at[0]:].any()
    cn, sn, pn, rn = sort.plan(ids, E, pad)
    for t, ref in ((idx, ids), (count, cn), (seg, sn), (pos, pn), (row_map, rn)):
        np.testing.assert_array_equal(t.cpu().numpy(), ref)
    v = to_np(x)
    src = np.where((rn >= 0)[:, None], v[np.maximum(rn, 0) // k], 0.0)
    np.testing.assert_array_equal(to_np(rows), src)
    # both of a token's rows are the token itself: y = x + x, d_rows = y / 2, dw = <y, x>, dx = 2 x
    np.testing.assert_array_equal(to_np(y), 2 * v)
    np.testing.assert_array_equal(to_np(dr), src)
    np.testing.assert_array_equal(to_np(dx), 2 * v)
    ref = (2 * v * v).sum(1)
    assert np.all(np.abs(to_np(dw) - ref[:, None]) <= (d + 1) * 2.0 ** -24 * ref[:, None])
    np.testing.assert_array_equal(to_np(back), fp4.rounded(src))
    wv, srcT = fp4.rounded(to_np(wn)).reshape(E, n, d), fp4.rounded(src.T)
    for e in range(E):
        r = slice(sn[e], sn[e] + cn[e])
        _check(to_np(c)[r], fp4.rounded(src)[r], wv[e], "f32", d)
        r = slice(sn[e], sn[e + 1])
        _check(to_np(g)[e], srcT[:, r], srcT[:, r], "f32", sn[e + 1] - sn[e])


def test_wgrad_of_the_longest_k(mb):
    """K = 2^31 - 1, the largest that the descriptor takes: segments at its beginning and
    at its far end (2^31 is no int)."""
    import torch
    k = (1 << 31) - 1
    d = mb.make_fp4_desc(1, k)
    codes = torch.zeros(mb.mlpblk_fp4_codes_size(d), dtype=torch.uint8, device="cuda")
    scales = torch.full((mb.mlpblk_fp4_scales_size(d),), 127, dtype=torch.uint8, device="cuda")
    end = (1 << 31) - 256
    codes[:128] = 0x22                                      # ones: 256 at the beginning, 64 at the end
    codes[end // 2 - 32:end // 2] = 0x22
    seg = torch.tensor([0, 512, 512, end], dtype=torch.int32, device="cuda")
    c = torch.full((3, 1, 1), 7.0, device="cuda")
    mb.mlpblk_fp4_wgrad_grouped(mb.make_fp4_matmul_desc(1, 1, k, "f32", experts=3, pad=256), codes, scales, codes, scales, seg, c)
    assert c.flatten().tolist() == [256.0, 0.0, 64.0]
    mb.mlpblk_fp4_wgrad_grouped(mb.make_fp4_matmul_desc(1, 1, k, "f32", True, 3, 256), codes, scales, codes, scales, seg, c)
    assert c.flatten().tolist() == [512.0, 0.0, 128.0]


# ------------------------------------- every kernel of the products, neighbours looked at

def _reaches(mb, desc, form, kernel):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert fp4_shapes.kernel(mb, desc, form, sms) == kernel


def _guarded(shape, dtype, fill):
    """A C of its own values (or NaN) in the middle of a larger buffer of sevens."""
    import torch
    n = int(np.prod(shape))
    whole = torch.full((n + 4096,), 7.0, dtype=_dt(dtype), device="cuda")
    c = whole[2048:2048 + n].view(shape)
    if fill is None:
        c.fill_(float("nan"))
    else:
        c.copy_(fill)
    return whole, c


def _untouched(whole):
    assert bool((whole[:2048] == 7.0).all()) and bool((whole[-2048:] == 7.0).all())


# A sum over a cluster adds up to eight parts, half a step each: four steps more, those of
# 128 more columns in _check's bound.
def _columns(k, kernel):
    return k + (128 if kernel in (2, 4, 8) else 0)


@pytest.mark.parametrize("shape,out,accumulate,kernel", fp4_shapes.DENSE)
def test_product_on_each_kernel(mb, shape, out, accumulate, kernel):
    import torch
    m, n, k = shape
    desc = fp4_shapes.dense_desc(mb, shape, out, accumulate)
    _reaches(mb, desc, 0, kernel)
    rng = np.random.default_rng(m + n + k + accumulate)
    qa, a = _quantized(mb, rng, m, k)
    qb, b = _quantized(mb, rng, n, k)
    base = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda() if accumulate else None
    whole, c = _guarded((m, n), out, base)
    mb.mlpblk_fp4_matmul(desc, qa.codes, qa.scales, qb.codes, qb.scales, c)
    _check(to_np(c), a, b, out, _columns(k, kernel), to_np(base) if accumulate else None)
    _untouched(whole)


@pytest.mark.parametrize("case,out,accumulate,kernel", fp4_shapes.GROUPED)
def test_grouped_product_on_each_kernel(mb, case, out, accumulate, kernel):
    import torch
    T, d, n, E, k, pad = case
    desc = fp4_shapes.grouped_desc(mb, case, out, accumulate)
    _reaches(mb, desc, 1, kernel)
    rng = np.random.default_rng(T + d + n)
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, pad, T, dead=(1,))
    assert s.rows == desc.m and count[1] == 0
    x, v = _draw(rng, (T, d), "bf16")
    qx = mb.Fp4Matrix(s.rows, d)
    qx.quantize(x, sort=s, gather=True)
    qw, w = _quantized(mb, rng, n, d, batch=E)
    base = torch.from_numpy(rng.standard_normal((s.rows, n)).astype(np.float32)).cuda()
    whole, c = _guarded((s.rows, n), out, base)
    before = to_np(c)
    mb.mlpblk_fp4_matmul_grouped(desc, qx.codes, qx.scales, qw.codes, qw.scales, s.count, s.seg, c)
    got = to_np(c)
    a = fp4.rounded(np.where((row_map >= 0)[:, None], v[np.maximum(row_map, 0) // k], 0.0))
    for e in range(E):
        r = slice(seg[e], seg[e] + count[e])
        if count[e]:
            _check(got[r], a[r], w[e], out, _columns(d, kernel), before[r] if accumulate else None)
        # padding rows: as they were, or zeros (times the weights, or added)
        p = slice(seg[e] + count[e], seg[e + 1])
        assert np.all((got[p] == before[p]) | (got[p] == 0.0))
    assert np.array_equal(got[seg[E]:], before[seg[E]:])
    _untouched(whole)


@pytest.mark.parametrize("case,accumulate,kernel", fp4_shapes.WGRAD)
def test_grouped_wgrad_on_each_kernel(mb, case, accumulate, kernel):
    """Expert 0 has no rows, expert 1 one block of 256, expert 2 two; the rest have the
    other tokens' rows."""
    import torch
    T, d, n, E, k = case
    desc = fp4_shapes.wgrad_desc(mb, case, accumulate)
    _reaches(mb, desc, 2, kernel)
    rng = np.random.default_rng(T + d + n)
    idx = rng.integers(3, E, (T, k)).astype(np.int32)
    idx[:200, 0], idx[200:500, 0] = 1, 2
    idx[rng.random((T, k)) < 0.01] = -1
    s = mb.MoeSort(T, d, E, k, 256)
    s.sort(torch.from_numpy(idx).cuda())
    count, seg, pos, row_map = sort.plan(idx, E, 256)
    assert count[0] == 0 and seg[2] - seg[1] == 256 and seg[3] - seg[2] == 512
    live = (row_map >= 0)[:, None]
    x, v = _draw(rng, (T, d), "bf16")
    dy, g = _draw(rng, (s.rows, n), "bf16")
    qx, qg = mb.Fp4Matrix(d, s.rows), mb.Fp4Matrix(n, s.rows)
    qx.quantize(x, sort=s, gather=True, transposed=True)
    qg.quantize(dy, sort=s, transposed=True)
    a = fp4.rounded(np.where(live, g, 0.0).T)
    b = fp4.rounded(np.where(live, v[np.maximum(row_map, 0) // k], 0.0).T)
    base = torch.from_numpy(rng.standard_normal((E, n, d)).astype(np.float32)).cuda() if accumulate else None
    whole, c = _guarded((E, n, d), "f32", base)
    mb.mlpblk_fp4_wgrad_grouped(desc, qg.codes, qg.scales, qx.codes, qx.scales, s.seg, c)
    got = to_np(c)
    for e in range(E):
        r = slice(seg[e], seg[e + 1])
        _check(got[e], a[:, r], b[:, r], "f32", _columns(int(seg[e + 1] - seg[e]), kernel), to_np(base)[e] if accumulate else None)
    assert np.array_equal(got[0], to_np(base)[0] if accumulate else np.zeros((n, d)))
    _untouched(whole)


# ------------------------------------------------------- through a sort, and captured

@pytest.mark.parametrize("act", ["none", "relu2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", [(45, 90, 5, 2, 128), (6, 301, 40, 2, 256), (37, 1032, 9, 3, 128), (70, 513, 4, 2, 1),
                                   (300, 40, 3, 1, 7)])
def test_quantize_through_a_sort_from_each_source(mb, shape, gather, dtype, act):
    """Both types, along rows and columns, buffers full of other bytes before: every byte
    of codes and scales is written, padding and unowned rows are zeros."""
    import torch
    T, d, E, k, pad = shape
    s, (count, seg, pos, row_map) = _routed(mb, T, d, E, k, pad, 7, dead=(2,))
    R = s.rows
    live = row_map >= 0
    x, v = _draw(np.random.default_rng(T + d), (T if gather else R, d), dtype)
    src = np.where(live[:, None], v[np.maximum(row_map, 0) // k] if gather else v, 0.0)
    if act == "relu2":                                      # squares in float32, as the operator says
        src = (np.maximum(src, 0.0).astype(np.float32) ** 2).astype(np.float64)
    if not gather:                                          # what no entry owns is not read
        x[torch.from_numpy(~live).cuda()] = float("nan")
    mask = 0xFF if act == "none" else 0x77                  # a square's zero has either sign
    for transposed in (False, True):
        q = mb.Fp4Matrix(*((d, R) if transposed else (R, d)))
        q.codes.fill_(0xAA)
        q.scales.fill_(0xAA)
        q.quantize(x, sort=s, gather=gather, transposed=transposed, act=act)
        packed, tiled = fp4.pack(*fp4.quantize(src.T if transposed else src))
        np.testing.assert_array_equal(_bytes(q.scales), tiled)
        np.testing.assert_array_equal(_bytes(q.codes) & mask, packed & mask)


def test_a_plan_not_made_yet(mb):
    """A MoeSort before its first sort: nothing is moved, gathered or multiplied."""
    import torch
    T, d, E, k = 33, 64, 3, 2
    for _ in range(2):
        junk = torch.full((1 << 20,), 5, dtype=torch.int32, device="cuda")
        del junk
        s = mb.MoeSort(T, d, E, k, 256)
        x = torch.randn(T, d, device="cuda").bfloat16()
        rows = torch.full((s.rows, d), 7.0, dtype=torch.bfloat16, device="cuda")
        s.permute(x, rows)
        assert bool((rows == 7.0).all())
        y = torch.empty_like(x)
        s.unpermute(rows, y, residual=x)
        assert torch.equal(y, x)
        q, w = mb.Fp4Matrix(s.rows, d), mb.Fp4Matrix(48, d, batch=E)
        q.codes.fill_(0xAA)
        q.scales.fill_(0xAA)
        q.quantize(x, sort=s, gather=True)
        assert not q.codes.any() and not q.scales.any()
        w.quantize(torch.randn(E * 48, d, device="cuda"))
        c = torch.full((s.rows, 48), 7.0, device="cuda")
        q.matmul_grouped(w, s, c)
        assert bool((c == 7.0).all())


def test_experts_captured_and_replayed_on_new_ids(mb):
    """The routed experts at 4 bits with the second layer's gradients, captured once and
    replayed on other tokens and ids: an expert loses all its rows and gains them again;
    each stage against the oracle on the stage's own input."""
    import torch
    T, d, F, E, k, pad = 200, 96, 288, 4, 2, 256
    rng = np.random.default_rng(22)
    bf = torch.bfloat16
    s = mb.MoeSort(T, d, E, k, pad)
    R = s.rows
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    x, dy = torch.zeros(T, d, dtype=bf, device="cuda"), torch.zeros(T, d, dtype=bf, device="cuda")
    p = torch.zeros(T, k, device="cuda")
    w1, b1 = _quantized(mb, rng, F, d, batch=E, wide=False)
    v2 = rng.standard_normal((E, d, F))
    pack = lambda v: _pack_batch(mb, v)
    (w2, b2), (w2t, b2t) = pack(v2), pack(v2.transpose(0, 2, 1))
    qx, qh, qo = mb.Fp4Matrix(R, d), mb.Fp4Matrix(R, F), mb.Fp4Matrix(R, d)
    qot, qht = mb.Fp4Matrix(d, R), mb.Fp4Matrix(F, R)
    h, o, do, dg = (torch.zeros(R, n, dtype=bf, device="cuda") for n in (F, d, d, F))
    y, dp, dw = torch.empty(T, d, dtype=bf, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(E, d, F, device="cuda")

    def step():
        s.sort(idx)
        qx.quantize(x, sort=s, gather=True)
        qx.matmul_grouped(w1, s, h)
        qh.quantize(h, sort=s, act="relu2")
        qh.matmul_grouped(w2, s, o)
        s.unpermute(o, y, weights=p, residual=x)
        s.unpermute_backward(dy, o, p, do, dp)
        qo.quantize(do, sort=s)
        qo.matmul_grouped(w2t, s, dg)
        qot.quantize(do, sort=s, transposed=True)
        qht.quantize(h, sort=s, act="relu2", transposed=True)
        qot.wgrad_grouped(qht, s, dw)

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for dead, eager in ((None, False), (1, False), (None, False), (3, True), (0, False)):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        if dead is not None:
            ids[ids == dead] = -1
        idx.copy_(torch.from_numpy(ids))
        for t in (x, dy):
            t.copy_(torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)))
        p.copy_(torch.from_numpy(rng.uniform(0.1, 1, (T, k)).astype(np.float32)))
        torch.cuda.synchronize()
        step() if eager else g.replay()
        torch.cuda.synchronize()
        count, seg, pos, row_map = sort.plan(ids, E, pad)
        for got, ref in zip((s.count, s.seg, s.pos, s.row_map), (count, seg, pos, row_map)):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        live = (row_map >= 0)[:, None]
        own = lambda t: np.where(live, to_np(t), 0.0)
        xv, dyv, pv, ov, dov = to_np(x), to_np(dy), to_np(p), own(o), own(do)
        a = fp4.rounded(np.where(live, xv[np.maximum(row_map, 0) // k], 0.0))
        hr = np.square(np.maximum(own(h), 0.0))
        aq, dq = fp4.rounded(hr), fp4.rounded(dov)
        dqt, hqt = fp4.rounded(dov.T), fp4.rounded(hr.T)
        for e in range(E):
            r, part = slice(seg[e], seg[e] + count[e]), slice(seg[e], seg[e + 1])
            if count[e]:
                _check(to_np(h)[r], a[r], b1[e], "bf16", d)
                _check(to_np(o)[r], aq[r], b2[e], "bf16", F)
                _check(to_np(dg)[r], dq[r], b2t[e], "bf16", d)
            _check(to_np(dw)[e], dqt[:, part], hqt[:, part], "f32", int(seg[e + 1] - seg[e]))
        ref, mag = sort.unpermute(ov, pos, pv, xv)
        assert np.all(np.abs(to_np(y) - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 2) * 2.0 ** -24 * mag)
        r_do, r_dp, mag = sort.unpermute_backward(dyv, ov, pos, row_map, pv)
        assert np.all(np.abs(dov - r_do) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(r_do))
        assert np.all(np.abs(to_np(dp) - r_dp) <= (d + 1) * 2.0 ** -24 * mag)


def _pack_batch(mb, v):
    """A batch of matrices quantised along their rows, and the values that they have."""
    import torch
    E, rows, cols = v.shape
    x = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).cuda()
    q = mb.Fp4Matrix(rows, cols, batch=E)
    q.quantize(x)
    return q, np.stack([fp4.rounded(to_np(x[e])) for e in range(E)])


def test_two_billion_rows(mb):
    """The most rows that a descriptor takes, quantised along rows and columns and read back."""
    import torch
    m = (1 << 31) - 1
    x = torch.arange(m, dtype=torch.int32, device="cuda").remainder_(7).to(torch.bfloat16)   # 0 .. 6, all but 5 E2M1 values
    x[x == 5] = -3.0
    q = mb.Fp4Matrix(m, 1)
    for transposed in (False, True):
        q.quantize(x.view(1, m) if transposed else x.view(m, 1), transposed=transposed)
        y = torch.full((m + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
        q.dequantize(y[:m].view(m, 1))
        assert torch.equal(y[:m], x) and bool((y[m:] == 9.0).all())
        q.codes[-16 * 4096:].fill_(0x77)                    # the second pass has these to mend


def test_products_of_two_billion_rows(mb):
    """The most rows that a descriptor takes, by both kernels, dense and as one expert's."""
    import torch
    m = (1 << 31) - 1
    x = torch.arange(m, dtype=torch.int32, device="cuda").remainder_(7).to(torch.bfloat16)
    x[x == 5] = -3.0
    q = mb.Fp4Matrix(m, 1)
    q.quantize(x.view(m, 1))
    w = mb.Fp4Matrix(1, 1)
    w.quantize(torch.full((1, 1), 4.0, device="cuda"))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ref = x * 4.0
    for out, kernel in (("bf16", "pair"), ("f32", 1)):
        d = mb.make_fp4_matmul_desc(m, 1, 1, out)
        assert fp4_shapes.kernel(mb, d, 0, sms) == kernel
        c = torch.full((m + 64,), 9.0, dtype=_dt(out), device="cuda")
        mb.mlpblk_fp4_matmul(d, q.codes, q.scales, w.codes, w.scales, c[:m])
        assert torch.equal(c[:m].bfloat16(), ref) and bool((c[m:] == 9.0).all())
        del c
    R, live = m + 1 - 128, m - 137
    count, seg = torch.tensor([live], dtype=torch.int32, device="cuda"), torch.tensor([0, R], dtype=torch.int32, device="cuda")
    for out, kernel in (("bf16", "pair"), ("f32", 1)):
        d = mb.make_fp4_matmul_desc(R, 1, 1, out, False, 1, 128)
        assert fp4_shapes.kernel(mb, d, 1, sms) == kernel
        c = torch.full((m,), 9.0, dtype=_dt(out), device="cuda")
        mb.mlpblk_fp4_matmul_grouped(d, q.codes, q.scales, w.codes, w.scales, count, seg, c[:R])
        assert torch.equal(c[:live].bfloat16(), ref[:live]) and bool((c[R:] == 9.0).all())
        pad = c[live:R].bfloat16()
        assert bool(((pad == 9.0) | (pad == ref[live:R])).all())
        del c


def test_calls_from_several_threads(mb):
    """Threads with their own streams and buffers, and one set of weights between them, in
    the middle of one another's calls (these run without the interpreter's lock)."""
    import threading
    import torch
    T, d, n, E, k, pad = 60, 128, 96, 4, 2, 128
    rng = np.random.default_rng(23)
    w, b = _quantized(mb, rng, n, d, batch=E, wide=False)
    work = []
    for i in range(4):
        ids = rng.integers(0, E, (T, k)).astype(np.int32)
        s = mb.MoeSort(T, d, E, k, pad)
        work.append(dict(ids=ids, idx=torch.from_numpy(ids).cuda(), s=s, x=_dev(rng.standard_normal((T, d)), "bf16"),
                         q=mb.Fp4Matrix(s.rows, d), c=torch.zeros(s.rows, n, device="cuda"),
                         back=torch.zeros(s.rows, d, device="cuda"), y=torch.zeros(T, n, dtype=torch.bfloat16, device="cuda"),
                         o=mb.MoeSort(T, n, E, k, pad), rows=torch.zeros(s.rows, n, dtype=torch.bfloat16, device="cuda"),
                         stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []
    start = threading.Barrier(len(work))

    def run(m):
        try:
            start.wait()
            with torch.cuda.stream(m["stream"]):
                for _ in range(100):
                    m["s"].sort(m["idx"])
                    m["o"].sort(m["idx"])
                    m["q"].quantize(m["x"], sort=m["s"], gather=True)
                    m["q"].matmul_grouped(w, m["s"], m["c"])
                    m["q"].matmul_grouped(w, m["s"], m["rows"])
                    m["q"].dequantize(m["back"])
                    m["o"].unpermute(m["rows"], m["y"])
                m["stream"].synchronize()
        except Exception as e:                              # shown by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=run, args=(m,)) for m in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for m in work:
        count, seg, pos, row_map = sort.plan(m["ids"], E, pad)
        src = np.where((row_map >= 0)[:, None], to_np(m["x"])[np.maximum(row_map, 0) // k], 0.0)
        a = fp4.rounded(src)
        np.testing.assert_array_equal(to_np(m["back"]), a)
        for e in range(E):
            r = slice(seg[e], seg[e] + count[e])
            _check(to_np(m["c"])[r], a[r], b[e], "f32", d)
            _check(to_np(m["rows"])[r], a[r], b[e], "bf16", d)
        ref, mag = sort.unpermute(to_np(m["rows"]), pos)
        assert np.all(np.abs(to_np(m["y"]) - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 1) * 2.0 ** -24 * mag)
