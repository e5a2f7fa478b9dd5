"""Pins of the token-sorting and MXFP4 oracles (CPU): values that the definitions
fix, the rounding's error bound, the byte layout spelled out, gradients against
central differences, and the refusals of the entry points."""

import ctypes

import numpy as np
import pytest

from oracle import fp4, sort


# ---------------------------------------------------------------------- MXFP4

def test_e2m1_values_and_ties():
    cases = {0.0: 0.0, 0.25: 0.0, 0.26: 0.5, 0.75: 1.0, 0.74: 0.5, 1.25: 1.0, 1.26: 1.5, 1.75: 2.0, 2.5: 2.0,
             2.51: 3.0, 3.5: 4.0, 5.0: 4.0, 5.01: 6.0, 6.0: 6.0, 7.9: 6.0}
    for v, q in cases.items():
        assert fp4.decode(fp4.e2m1(np.array([v])))[0] == q, v
        assert fp4.decode(fp4.e2m1(np.array([-v])))[0] == -q, -v


@pytest.mark.parametrize("top,byte", [(6.0, 127), (4.0, 127), (3.99, 126), (1.0, 125), (8.0, 128), (0.0, 0),
                                      (2.0 ** -126, 0), (2.0 ** -124, 1), (2.0 ** 127, 252), (np.inf, 255), (np.nan, 255)])
def test_scale_byte(top, byte):
    v = np.zeros((1, 32))
    v[0, 7] = -top
    assert fp4.quantize(v)[1][0, 0] == byte


def test_rounding_error_bound():
    v = np.random.default_rng(0).standard_normal((64, 256)) * 3.0
    c, s = fp4.quantize(v)
    q = fp4.values(c, s, 256)
    scale = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    # half a step: 1/4, 1/2 or 1 scale by binade; saturation cuts [6, 8) scales down to 6
    assert np.all(np.abs(q - v) <= np.where(np.abs(v) < 2 * scale, 0.25, np.where(np.abs(v) < 4 * scale, 0.5, 2.0)) * scale)


def test_layout_byte_by_byte():
    rng = np.random.default_rng(1)
    rows, cols = 200, 300
    codes, sb = fp4.quantize(rng.standard_normal((rows, cols)))
    packed, tiled = fp4.pack(codes, sb)
    assert packed.size == rows * 10 * 16 and tiled.size == 2 * 4 * 512
    for r, c in ((0, 0), (199, 299), (130, 131), (64, 33)):
        assert packed[r * 160 + c // 2] >> (4 * (c % 2)) & 15 == codes[r, c]
        b = c // 32
        assert tiled[(r // 128 * 4 + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] == sb[r, b]


# -------------------------------------------------------------------- sorting

def test_plan_by_hand():
    idx = np.array([[1, 0], [1, -1], [2, 1], [1, 1]])
    count, seg, pos, row_map = sort.plan(idx, 4, 4)
    assert count.tolist() == [1, 5, 1, 0] and seg.tolist() == [0, 4, 12, 16, 16]
    assert pos.tolist() == [[4, 0], [5, -1], [12, 6], [7, 8]]
    assert row_map[:16].tolist() == [1, -1, -1, -1, 0, 2, 5, 6, 7, -1, -1, -1, 4, -1, -1, -1]
    assert len(row_map) == 8 + 4 * 3 and np.all(row_map[16:] == -1)


def test_gradients_against_differences():
    rng = np.random.default_rng(2)
    T, d, E, k = 5, 6, 3, 2
    idx = rng.integers(-1, E, (T, k))
    _, _, pos, row_map = sort.plan(idx, E, 2)
    R = len(row_map)
    rows, w = rng.standard_normal((R, d)), rng.uniform(0.1, 1, (T, k))
    x, dy, g = rng.standard_normal((T, d)), rng.standard_normal((T, d)), rng.standard_normal((R, d))
    live = row_map >= 0
    d_rows, dw, _ = sort.unpermute_backward(dy, rows, pos, row_map, w)
    dx = sort.permute_backward(np.where(live[:, None], g, 0.0), pos)
    h = 1e-6

    def check(f, at, grad):
        for ij in np.ndindex(at.shape):
            keep = at[ij]
            at[ij] = keep + h
            up = f()
            at[ij] = keep - h
            down = f()
            at[ij] = keep
            assert abs((up - down) / (2 * h) - grad[ij]) < 1e-7

    check(lambda: float(np.sum(sort.unpermute(rows, pos, w, x)[0] * dy)), rows, d_rows)
    check(lambda: float(np.sum(sort.unpermute(rows, pos, w, x)[0] * dy)), w, dw)
    check(lambda: float(np.sum(sort.permute(x, row_map, k)[live] * g[live])), x, dx)


# ------------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def mb():
    import __graft_entry__
    __graft_entry__.build()
    import mlp_block_backprop_gb300
    return mlp_block_backprop_gb300


def _addresses(n):
    return [0x10000 * (i + 1) for i in range(n)]  # aligned, never dereferenced


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(width=0), dict(experts=0), dict(experts=257), dict(top_k=0),
                                dict(top_k=257), dict(pad=0), dict(pad=1025), dict(tokens=1 << 31), dict(width=1 << 30)])
def test_sort_desc_refusals(mb, kw):
    base = dict(tokens=10, width=64, experts=4, top_k=2, pad=128)
    assert mb.mlpblk_moe_sort_rows(mb.make_sort_desc(**base)) == sort.rows_bound(10, 2, 4, 128)
    bad = mb.make_sort_desc(**{**base, **kw})
    assert mb.mlpblk_moe_sort_rows(bad) == -1
    p = _addresses(9)
    b = ctypes.byref(bad)
    assert mb.lib.mlpblk_moe_sort(b, *p[:5], None) == mb.MLPBLK_EINVAL
    assert mb.lib.mlpblk_moe_permute(b, *p[:5], None) == mb.MLPBLK_EINVAL
    assert mb.lib.mlpblk_moe_unpermute_backward(b, *p[:8], None) == mb.MLPBLK_EINVAL


def test_sort_argument_refusals(mb):
    d = mb.make_sort_desc(10, 64, 4, 2, 128)
    b = ctypes.byref(d)
    assert mb.mlpblk_moe_sort_rows(mb.SortDesc(10, 64, 4, 2, 128, 7)) == -1
    assert mb.lib.mlpblk_moe_permute(ctypes.byref(mb.SortDesc(10, 64, 4, 2, 128, 7)), *_addresses(5), None) == mb.MLPBLK_ENOTSUP
    for name, n, out, ins in (("mlpblk_moe_permute", 5, 4, (0,)), ("mlpblk_moe_permute_backward", 3, 2, (0,)),
                              ("mlpblk_moe_unpermute", 5, 4, (0,)), ("mlpblk_moe_unpermute_backward", 8, 6, (0, 1)),
                              ("mlpblk_moe_sort", 5, 3, (0,))):
        f = getattr(mb.lib, name)
        p = _addresses(n)
        for i in range(n):
            q = list(p)
            q[i] += 8
            assert f(b, *q, None) == mb.MLPBLK_EINVAL, (name, i)  # misaligned
        q = list(p)
        q[0] = None
        assert f(b, *q, None) == mb.MLPBLK_EINVAL
        for i in ins:
            q = list(p)
            q[out] = q[i]
            assert f(b, *q, None) == mb.MLPBLK_EINVAL, (name, "alias", i)
    empty = ctypes.byref(mb.make_sort_desc(0, 64, 4, 2, 128))
    assert mb.mlpblk_moe_sort_rows(mb.make_sort_desc(0, 64, 4, 2, 128)) == 0
    assert mb.lib.mlpblk_moe_permute(empty, *[None] * 5, None) == mb.MLPBLK_OK
    assert mb.lib.mlpblk_moe_unpermute(empty, *[None] * 5, None) == mb.MLPBLK_OK
    assert mb.lib.mlpblk_moe_unpermute_backward(empty, *[None] * 8, None) == mb.MLPBLK_OK


def _spans(mb):
    """Every entry point with its arguments' sizes in bytes, which of them are outputs, and
    a call of it."""
    at = ctypes.byref
    T, w, E, k, pad = 10, 64, 5, 2, 128
    s = mb.make_sort_desc(T, w, E, k, pad)
    R, n = mb.mlpblk_moe_sort_rows(s), T * k
    x, r, c, g = 2 * T * w, 2 * R * w, 4 * E, 4 * (E + 1)
    yield "mlpblk_moe_sort", (at(s),), [4 * n, c, g, 4 * n, 4 * R], (1, 2, 3, 4)
    yield "mlpblk_moe_permute", (at(s),), [x, 4 * n, c, g, r], (4,)
    yield "mlpblk_moe_permute_backward", (at(s),), [r, 4 * n, x], (2,)
    yield "mlpblk_moe_unpermute", (at(s),), [r, 4 * n, 4 * n, x, x], (4,)
    yield "mlpblk_moe_unpermute_backward", (at(s),), [x, r, 4 * n, c, g, 4 * n, r, 4 * n], (6, 7)
    size = lambda rows, cols, b=1: [rows * b * -(-cols // 32) * 16, -(-rows // 128) * -(-cols // 256) * 1024 * b]
    for tr, b in ((0, 1), (1, 1), (0, 3)):
        q = mb.make_fp4_desc(40, 300, b, transposed=tr)
        yield "mlpblk_fp4_quantize", (at(q),), [2 * b * 40 * 300, None, None] + size(40, 300, b), (3, 4)
    for tr in (0, 1):
        q = mb.make_fp4_desc(40, 300, dtype="f32", transposed=tr, source_rows=7)
        yield "mlpblk_fp4_quantize", (at(q),), [4 * 7 * (40 if tr else 300), 4 * (300 if tr else 40), 2] + size(40, 300), (3, 4)
        yield "mlpblk_fp4_quantize", (at(q),), [4 * 40 * 300, 4 * (300 if tr else 40), 0] + size(40, 300), (3, 4)
    yield "mlpblk_fp4_dequantize", (at(mb.make_fp4_desc(40, 300, 2)),), size(40, 300, 2) + [2 * 2 * 40 * 300], (2,)
    yield "mlpblk_fp4_matmul", (at(mb.make_fp4_matmul_desc(40, 50, 300, "f32")),), size(40, 300) + size(50, 300) + [4 * 40 * 50], (4,)
    yield ("mlpblk_fp4_matmul_grouped", (at(mb.make_fp4_matmul_desc(256, 50, 300, experts=E, pad=128)),),
           size(256, 300) + size(50, 300, E) + [c, g, 2 * 256 * 50], (6,))
    yield ("mlpblk_fp4_wgrad_grouped", (at(mb.make_fp4_matmul_desc(40, 50, 512, "f32", experts=E, pad=256)),),
           size(40, 512) + size(50, 512) + [g, 4 * E * 40 * 50], (5,))


def test_outputs_that_share_bytes_are_refused(mb):
    """Each output laid over the end and over the beginning of every other argument, and
    inside it.  (No call here would be accepted: the addresses are never used.)"""
    for name, desc, sizes, outs in _spans(mb):
        f = getattr(mb.lib, name)
        buffers = [i for i, n in enumerate(sizes) if n is not None and not (name == "mlpblk_fp4_quantize" and i == 2)]
        base = [None if n is None else (n if i not in buffers else 0x10000000 * (i + 1)) for i, n in enumerate(sizes)]
        if name == "mlpblk_fp4_quantize" and sizes[2] is None:
            base[2] = 0
        for o in outs:
            for i in buffers:
                if i == o:
                    continue
                inside = (sizes[i] - 1) // 16 * 16
                for at in (base[i], base[i] + inside, base[i] - (sizes[o] - 1) // 16 * 16, base[i] + inside // 32 * 16):
                    if name == "mlpblk_moe_unpermute" and i == 3 and at == base[i]:
                        continue                           # y may be residual itself
                    q = list(base)
                    q[o] = at
                    assert f(*desc, *q, None) == mb.MLPBLK_EINVAL, (name, "argument", o, "over", i, hex(at))


@pytest.mark.parametrize("shape", [(10, 4, 2, 128), (5, 200, 3, 1), (0, 4, 2, 16)])
def test_a_plan_not_made_yet_selects_nothing(mb, shape):
    """The plan's buffers of a new MoeSort, in memory that held something else before."""
    torch = pytest.importorskip("torch")
    T, E, k, pad = shape
    for _ in range(3):
        keep = [torch.full((max(n, 1),), 7, dtype=torch.int32) for n in (T * k, sort.rows_bound(T, k, E, pad))]
        del keep
        s = mb.MoeSort(T, 64, E, k, pad, device="cpu")
        ref = sort.plan(np.full((T, k), -1), E, pad)
        for got, want in zip((s.count, s.seg, s.pos, s.row_map), ref):
            np.testing.assert_array_equal(got.numpy(), want)


def test_fp4_sizes_and_refusals(mb):
    size = lambda r, c, b=1: (mb.mlpblk_fp4_codes_size(mb.make_fp4_desc(r, c, b)),
                              mb.mlpblk_fp4_scales_size(mb.make_fp4_desc(r, c, b)))
    assert size(1, 1) == (16, 1024)
    assert size(129, 257, 3) == (3 * 129 * 144, 3 * 2 * 4 * 512)
    assert size(0, 64) == (0, 0)
    q = lambda d, x=0x10000, rm=None, div=0, c=0x20000, s=0x30000: mb.lib.mlpblk_fp4_quantize(ctypes.byref(d), x, rm, div, c, s, None)
    good = mb.make_fp4_desc(8, 64)
    for bad in (mb.make_fp4_desc(-1, 64), mb.make_fp4_desc(8, -1), mb.make_fp4_desc(8, 64, 0), mb.make_fp4_desc(1 << 30, 64, 2),
                mb.make_fp4_desc(8, 1 << 31), mb.make_fp4_desc(1 << 16, (1 << 31) - 1), mb.make_fp4_desc(1, 257, 1 << 28)):
        assert q(bad) == mb.MLPBLK_EINVAL
    assert q(mb.Fp4Desc(8, 64, 1, 3, 0, 0)) == mb.MLPBLK_ENOTSUP
    assert q(mb.make_fp4_desc(8, 64, act=2)) == mb.MLPBLK_ENOTSUP
    assert q(mb.Fp4Desc(8, 64, 1, mb.MLPBLK_BF16, 2, 0)) == mb.MLPBLK_EINVAL
    assert q(good, x=None) == q(good, x=0x10008) == q(good, rm=0x40004) == q(good, c=0x10000) == mb.MLPBLK_EINVAL
    assert q(good, div=-1) == mb.MLPBLK_EINVAL
    assert q(mb.make_fp4_desc(8, 64, 2), rm=0x40000) == mb.MLPBLK_EINVAL          # a row map takes one matrix
    assert q(mb.make_fp4_desc(0, 64), x=None) == q(mb.make_fp4_desc(8, 0), x=None) == mb.MLPBLK_OK
    dq = lambda d, y=0x30000: mb.lib.mlpblk_fp4_dequantize(ctypes.byref(d), 0x10000, 0x20000, y, None)
    assert dq(mb.make_fp4_desc(8, 64, transposed=True)) == dq(mb.make_fp4_desc(8, 64, act=1)) == mb.MLPBLK_ENOTSUP
    assert dq(good, 0x10000) == dq(good, 0x30004) == mb.MLPBLK_EINVAL


def test_fp4_gather_needs_the_sources_rows(mb):
    """A row map that gathers is taken only with the source's row count: the map's
    values are device data, and nothing else bounds the rows that are read."""
    q = lambda d, rm=0x40000, div=2: mb.lib.mlpblk_fp4_quantize(ctypes.byref(d), 0x10000, rm, div, 0x20000, 0x30000, None)
    for n in (0, -1, 1 << 31):
        for tr in (False, True):
            assert q(mb.make_fp4_desc(8, 64, transposed=tr, source_rows=n)) == mb.MLPBLK_EINVAL
    assert q(mb.make_fp4_desc(0, 64)) == q(mb.make_fp4_desc(8, 0)) == mb.MLPBLK_OK    # nothing is read
    assert mb.mlpblk_fp4_codes_size(mb.make_fp4_desc(8, 64, source_rows=-1)) == 8 * 32  # of no meaning elsewhere


def test_version_tells_of_the_descriptors_field(mb):
    assert mb.mlpblk_version() >= 101 and mb.Fp4Desc._fields_[-1][0] == "source_rows" and ctypes.sizeof(mb.Fp4Desc) == 40


def test_fp4_product_refusals(mb):
    p = _addresses(5)
    mm = lambda d, a=p: mb.lib.mlpblk_fp4_matmul(ctypes.byref(d), *a, None)
    D = mb.make_fp4_matmul_desc
    for bad in (D(-1, 8, 8), D(8, 0, 8), D(8, 8, 0), D(1 << 31, 8, 8), D(8, 8, 8, experts=2), D(8, 8, 8, pad=128),
                D(8, 8, 8, max_rows=4), mb.Fp4MatmulDesc(8, 8, 8, mb.MLPBLK_FP32, 2, 0, 0, 0), D((1 << 31) - 1, (1 << 31) - 1, 8)):
        assert mm(bad) == mb.MLPBLK_EINVAL
    assert mm(D(8, 8, 8, accumulate=True)) == mb.MLPBLK_ENOTSUP                   # bf16 sums are not kept
    assert mm(mb.Fp4MatmulDesc(8, 8, 8, 9, 0, 0, 0, 0)) == mb.MLPBLK_ENOTSUP
    for i in range(5):
        q = list(p)
        q[i] += 8
        assert mm(D(8, 8, 8), q) == mb.MLPBLK_EINVAL
    for i in range(4):
        q = list(p)
        q[4] = q[i]
        assert mm(D(8, 8, 8), q) == mb.MLPBLK_EINVAL
    assert mm(D(0, 8, 8), [None] * 5) == mb.MLPBLK_OK
    g = _addresses(7)
    gr = lambda d, a=g: mb.lib.mlpblk_fp4_matmul_grouped(ctypes.byref(d), *a, None)
    assert gr(D(256, 8, 8, experts=0, pad=128)) == gr(D(256, 8, 8, experts=257, pad=128)) == mb.MLPBLK_EINVAL
    assert gr(D(256, 8, 8, experts=2, pad=64)) == mb.MLPBLK_ENOTSUP
    assert gr(D(256, 1 << 30, 8, experts=2, pad=128)) == mb.MLPBLK_EINVAL
    assert gr(D(256, 8, 8, experts=2, pad=128), g[:5] + [None, g[6]]) == mb.MLPBLK_EINVAL   # seg
    wg = lambda d: mb.lib.mlpblk_fp4_wgrad_grouped(ctypes.byref(d), *_addresses(6), None)
    assert wg(D(8, 8, 256, experts=2, pad=128)) == mb.MLPBLK_ENOTSUP
    assert wg(D(1 << 30, 8, 256, experts=2, pad=256)) == mb.MLPBLK_EINVAL
    assert wg(D(8, 8, 256, experts=2, pad=256, max_rows=3)) == mb.MLPBLK_EINVAL


def test_binding_refuses_wrong_tensors(mb):
    torch = pytest.importorskip("torch")
    with pytest.raises(mb.MlpBlkError):                       # not a CUDA tensor
        mb._operand(torch.zeros(4), "f", "x", torch.float32, 4, 0)
    assert mb._operand(None, "f", "x", torch.float32, 4, 0) is None
    with pytest.raises(mb.MlpBlkError):
        mb.make_sort_desc(1, 1, 1, 1, dtype="f16")
    with pytest.raises(mb.MlpBlkError):
        mb.Fp4Matrix(4, 64, codes=torch.zeros(3, dtype=torch.uint8), scales=torch.zeros(1024, dtype=torch.uint8), device="cpu")


def test_both_ways_into_the_library_agree(mb):
    """The CPython entry points (where built) and ctypes give the same refusals, and the
    former check their argument count and types before they call."""
    slow = {n: mb._Calls._ctypes("mlpblk_" + n) for n in ("moe_sort", "fp4_quantize", "fp4_matmul", "fp4_wgrad_grouped")}
    sort, fp4, mm = mb.make_sort_desc(10, 64, 4, 2), mb.make_fp4_desc(8, 64), mb.make_fp4_matmul_desc(8, 8, 256, experts=2, pad=128)
    at = ctypes.addressof
    cases = [("moe_sort", (at(sort), None, 0x10000, 0x20000, 0x30000, 0x40000, None)),
             ("moe_sort", (at(sort), 0x10000, 0x20008, 0x30000, 0x40000, 0x50000, None)),
             ("fp4_quantize", (at(fp4), 0x10000, None, -1, 0x20000, 0x30000, None)),
             ("fp4_quantize", (at(fp4), 0x10000, None, 0, 0x10000, 0x30000, None)),
             ("fp4_matmul", (at(mm),) + tuple(_addresses(5)) + (None,)),
             ("fp4_wgrad_grouped", (at(mm),) + tuple(_addresses(6)) + (None,))]
    for name, args in cases:
        rc = slow[name](*args)
        assert rc in (mb.MLPBLK_EINVAL, mb.MLPBLK_ENOTSUP)
        assert getattr(mb._calls, name)(*args) == rc, name
    if mb._calls.native:
        with pytest.raises(TypeError):
            mb._calls.fp4_quantize(at(fp4), 0x10000)
        with pytest.raises(TypeError):
            mb._calls.fp4_quantize(at(fp4), "x", None, 0, 0x20000, 0x30000, None)


def test_descriptors_of_first_calls_from_several_threads(mb):
    """Threads that make the first calls with different options on one matrix: each
    kept descriptor is its key's, also where threads change over between any two
    steps of making one (`_kept` below yields there)."""
    import threading
    import time
    torch = pytest.importorskip("torch")
    u8 = dict(dtype=torch.uint8, device="cpu")

    class Yielding(list):
        def append(self, d):
            super().append(d)
            time.sleep(0.01)

    for _ in range(3):
        q = mb.Fp4Matrix(4, 64, codes=torch.zeros(4 * 32, **u8), scales=torch.zeros(1024, **u8), device="cpu")
        q._kept = Yielding()
        keys = [(dt, tr, act, n) for dt in (torch.bfloat16, torch.float32) for tr in (False, True)
                for act in ("none", "relu2") for n in (0, 9)]
        got = {}
        start = threading.Barrier(2 * len(keys))

        def first_call(i, key):
            start.wait()
            got[i] = q._desc(*key)

        threads = [threading.Thread(target=first_call, args=(i, k)) for i, k in enumerate(keys * 2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for i, (dt, tr, act, n) in enumerate(keys * 2):
            assert got[i] == q._descs[(dt, tr, act, n)]
            d = mb.Fp4Desc.from_address(got[i])
            assert (d.rows, d.cols, d.batch) == (4, 64, 1)
            assert (d.dtype, d.transposed, d.act, d.source_rows) == (
                mb.MLPBLK_BF16 if dt is torch.bfloat16 else mb.MLPBLK_FP32, int(tr), int(act == "relu2"), n)


_STUB = """
#include <stdint.h>
#include <time.h>
#include "mlpblk.h"
volatile int stub_entered = 0, stub_release = 0;
/* waits up to 5 s for another thread to set stub_release: 0 where it did, else 1 */
static int waited(void) {
    struct timespec t0, t;
    clock_gettime(CLOCK_MONOTONIC, &t0);
    stub_entered = 1;
    do clock_gettime(CLOCK_MONOTONIC, &t);
    while (!stub_release && t.tv_sec - t0.tv_sec < 5);
    return stub_release ? 0 : 1;
}
"""


def test_native_calls_let_other_threads_run(mb, tmp_path):
    """The CPython entry points around stand-ins that return only once another Python
    thread has run: each is entered without the interpreter's lock."""
    import os
    import re
    import subprocess
    import sys
    import sysconfig
    if not mb._calls.native:
        pytest.skip("built without Python's headers")
    root = os.path.dirname(os.path.dirname(os.path.abspath(mb.__file__)))
    src = os.path.join(root, "mlp_block_backprop_gb300", "csrc", "pycalls.c")
    names = re.findall(r"^CALL\((\w+), (\d+),", open(src).read(), flags=re.M)
    assert len(names) >= 10
    header = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "mlpblk.h")).read(), flags=re.S)
    stubs = ""
    for name, _ in names:
        params = re.search(r"int mlpblk_%s\(([^;]*?)\);" % name, header, flags=re.S).group(1)
        stubs += "int mlpblk_%s(%s) { return waited(); }\n" % (name, params)
    c = tmp_path / "stub.c"
    c.write_text(_STUB + stubs)
    inc = sysconfig.get_paths()["include"]
    out = str(tmp_path / "_mlpblk_calls.so")
    r = subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-I", inc, "-I", os.path.join(root, "include"), "-I", os.path.dirname(src),
                        src, str(c), "-o", out, "-Wl,-Bsymbolic"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = f"""
import ctypes, importlib.machinery, importlib.util, threading, time
spec = importlib.util.spec_from_file_location("_mlpblk_calls", {out!r})
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
stub = ctypes.CDLL({out!r})
entered, release = ctypes.c_int.in_dll(stub, "stub_entered"), ctypes.c_int.in_dll(stub, "stub_release")
for name, n in {[(n, int(k)) for n, k in names]!r}:
    entered.value = release.value = 0
    def other():
        while not entered.value:
            time.sleep(0.001)
        release.value = 1
    t = threading.Thread(target=other)
    t.start()
    rc = getattr(m, "mlpblk_" + name)(*[16] * n)
    t.join()
    assert rc == 0, name
"""
    r = subprocess.run([sys.executable, "-c", run], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr


def test_native_calls_belong_to_one_interpreter(mb, tmp_path):
    """The module's file name carries the interpreter's ABI tag; one without a tag, or of
    another interpreter, is not loaded: the calls then go through ctypes."""
    import importlib.machinery
    import os
    import shutil
    import subprocess
    import sys
    if not mb._calls.native:
        pytest.skip("built without Python's headers")
    suffix = importlib.machinery.EXTENSION_SUFFIXES[0]
    here = os.path.dirname(os.path.abspath(mb.__file__))
    built = os.path.join(here, "_mlpblk_calls" + suffix)
    assert "cpython" in suffix and os.path.exists(built)
    pkg = tmp_path / "mlp_block_backprop_gb300"
    pkg.mkdir()
    for name in ("__init__.py", "libmlpblk.so"):
        shutil.copy(os.path.join(here, name), pkg / name)
    run = "import mlp_block_backprop_gb300 as mb; print(mb.__file__, mb._calls.native)"
    for name, native in (("_mlpblk_calls.so", False), ("_mlpblk_calls.cpython-39-none.so", False), ("_mlpblk_calls" + suffix, True)):
        shutil.copy(built, pkg / name)
        r = subprocess.run([sys.executable, "-c", run], capture_output=True, text=True, cwd=tmp_path,
                           env={**os.environ, "PYTHONPATH": str(tmp_path)})
        assert r.returncode == 0 and r.stdout.split() == [str(pkg / "__init__.py"), str(native)], (name, r)


def test_a_new_library_leaves_no_other_interpreters_module(tmp_path, monkeypatch):
    """A module built against the library before this one does not stay behind."""
    import __graft_entry__
    build = __graft_entry__._build_script()
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    for name in ("_mlpblk_calls.so", "_mlpblk_calls.cpython-39-none.so", "libmlpblk.so", "other.so"):
        (tmp_path / name).write_bytes(b"")
    build._remove_calls()
    assert sorted(f.name for f in tmp_path.iterdir()) == ["libmlpblk.so", "other.so"]


@pytest.mark.parametrize("sms", [148, 152])
def test_product_shapes_reach_the_kernels_they_are_for(mb, sms):
    import fp4_shapes as f
    got = [(c, f.kernel(mb, f.dense_desc(mb, *c[:3]), 0, sms)) for c in f.DENSE]
    got += [(c, f.kernel(mb, f.grouped_desc(mb, *c[:3]), 1, sms)) for c in f.GROUPED]
    got += [(c, f.kernel(mb, f.wgrad_desc(mb, *c[:2]), 2, sms)) for c in f.WGRAD]
    assert not [(c, k) for c, k in got if k != c[-1]]
    # every instantiation of the two kernels (output type, += and the store of C) is among them
    kinds = {(c[1], c[2], "split" if k in (2, 4, 8) else k) for c, k in got[:len(f.DENSE)]}
    assert {(o, a, k) for o, a in (("bf16", False), ("f32", False), ("f32", True)) for k in ("tma", "pair", "split")} <= kinds


def test_product_kernel_refusals(mb):
    D = mb.make_fp4_matmul_desc
    f = mb.mlpblk_fp4_product_kernel
    assert f(D(8, 8, 8), 0, 152) == 1
    assert f(D(8, 8, 8), 3, 152) == f(D(8, 8, 8), -1, 152) == f(D(8, 8, 8), 0, 0) == f(D(0, 8, 8), 0, 152) == -1
    assert f(D(8, 8, 8), 1, 152) == f(D(8, 0, 8), 0, 152) == f(D(8, 8, 0, experts=2, pad=256), 2, 152) == -1
    assert mb.lib.mlpblk_fp4_product_kernel(None, 0, 152) == -1


def test_limits_as_documented(mb):
    """rows * batch, experts * n and tokens * top_k are taken up to 2^31 - 1, whether or not
    the factors divide 2^31."""
    size = lambda *a: mb.mlpblk_fp4_codes_size(mb.make_fp4_desc(*a))
    top = (1 << 31) - 1
    for rows, batch in ((top, 1), ((1 << 30) + 1, 1), (715827882, 3), (1 << 30, 1)):
        assert size(rows, 1, batch) == rows * batch * 16
    assert size(1 << 31, 1) == size(715827883, 1, 3) == size(1 << 62, 1, 4) == 0
    D, f = mb.make_fp4_matmul_desc, mb.mlpblk_fp4_product_kernel
    assert f(D(128, 715827882, 1, experts=3, pad=128), 1, 152) > 0 and f(D(128, 715827883, 1, experts=3, pad=128), 1, 152) == -1
    assert f(D(715827882, 1, 256, experts=3, pad=256), 2, 152) > 0 and f(D(715827883, 1, 256, experts=3, pad=256), 2, 152) == -1
    rows = lambda t, k, pad=1: mb.mlpblk_moe_sort_rows(mb.make_sort_desc(t, 1, 1, k, pad))
    assert rows(715827881, 3) == 715827881 * 3 and rows(715827882, 3) == rows(1 << 31, 1) == rows((1 << 31) - 1, 256) == -1


def test_two_interpreters_keep_their_modules(tmp_path, monkeypatch):
    """A second interpreter's build beside a library that is up to date makes its own module
    and leaves the library and the first one's alone."""
    import __graft_entry__
    build = __graft_entry__._build_script()
    lib, mine, other = (tmp_path / n for n in ("libmlpblk.so", "_mlpblk_calls.mine.so", "_mlpblk_calls.cpython-39-none.so"))
    lib.write_bytes(b"library")
    other.write_bytes(b"other")
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "CALLS", str(mine))
    monkeypatch.setattr(build, "_newest_input_mtime", lambda: 0.0)
    monkeypatch.setattr(build, "_python_headers", lambda: str(tmp_path))
    monkeypatch.setattr(build, "nvcc", lambda: pytest.fail("the library is up to date"))
    monkeypatch.setattr(build, "_build_calls", lambda: mine.write_bytes(b"mine"))
    assert build.build_library() == str(lib) and mine.read_bytes() == b"mine" and other.read_bytes() == b"other"
    mine.write_bytes(b"kept")
    assert build.build_library() == str(lib) and mine.read_bytes() == b"kept"
