"""The work of the token-sorting and MXFP4 operators, as cases that can be timed.

Each case is one pass as a program around the block would make it:

  dispatch  tokens sorted by expert, their rows brought into that order, the
            experts' output rows weighted and added back per token; with the
            gradients of both moves
  quant     a matrix rounded to MXFP4 (blocks of 32 values along a row share one
            power-of-two scale, each value is kept in 4 bits) and read back
  product   activations rounded to MXFP4 and multiplied with MXFP4 weights; a
            training pass adds the gradients of the activations and the weights
  experts   the same product for tokens sorted by expert, each expert with its own
            weights; a training pass adds both gradients

With ``own`` false, ``run`` computes a case in plain torch operations in 32 bits;
with ``own`` true it calls mlp_block_backprop_gb300.
"""

import math

import numpy as np
import torch

own = False

BLOCK = 32            # values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one step of serving 8 sequences through 8 experts: latency alone
        dict(name="dispatch_decode", op="dispatch", tokens=8, width=2048, experts=8, top_k=2, pad=128,
             dtype="bf16", grad=False, skew=False),
        # a training microbatch of the large block's width, forward and backward
        dict(name="dispatch_train", op="dispatch", tokens=16384, width=4096, experts=8, top_k=2, pad=256,
             dtype="bf16", grad=True, skew=False),
        # many small experts, uneven load, some slots that choose nothing, odd sizes, float32, no padding
        dict(name="dispatch_ragged", op="dispatch", tokens=4097, width=1001, experts=60, top_k=6, pad=1,
             dtype="f32", grad=True, skew=True),
        # the activations of 8 tokens on their way into a product
        dict(name="quant_tokens", op="quant", rows=8, cols=4096, dtype="bf16", transposed=False, act="none"),
        # the hidden layer of the large block: ReLU^2 applied as it is read
        dict(name="quant_hidden", op="quant", rows=16384, cols=16384, dtype="bf16", transposed=False, act="relu2"),
        # a float32 gradient of odd sizes, rounded along its columns for a weight gradient
        dict(name="quant_columns", op="quant", rows=1031, cols=4095, dtype="f32", transposed=True, act="none"),
        # one token through the large block's up projection: bound by the weights' bytes
        dict(name="product_token", op="product", m=1, n=16384, k=4096, out="bf16", train=False),
        # a ragged batch, nothing a multiple of a tile, float32 out
        dict(name="product_odd", op="product", m=333, n=1000, k=1031, out="f32", train=False),
        # the large block's up projection, a microbatch of 8192 tokens, forward and backward
        dict(name="product_train", op="product", m=8192, n=16384, k=4096, out="bf16", train=True),
        # serving 8 tokens through 8 experts: bound by the experts' weights
        dict(name="experts_decode", op="experts", tokens=8, width=2048, out_width=8192, experts=8, top_k=2,
             pad=128, train=False, skew=False),
        # a prompt through many small experts of odd widths, uneven load, experts without a token
        dict(name="experts_ragged", op="experts", tokens=1500, width=1000, out_width=776, experts=60, top_k=4,
             pad=128, train=False, skew=True),
        # a training microbatch of the wide block's widths through 8 experts, forward and backward
        dict(name="experts_train", op="experts", tokens=8192, width=2048, out_width=8192, experts=8, top_k=2,
             pad=256, train=True, skew=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above."""
    while True:
        op = rng.choice(["dispatch", "quant", "product", "experts"])
        if op == "dispatch":
            experts = _log_int(rng, 2, 256)
            top_k = rng.randint(1, min(8, experts))
            c = dict(op=op, tokens=_log_int(rng, 1, 16384), width=_log_int(rng, 64, 4096), experts=experts,
                     top_k=top_k, pad=rng.choice([1, 16, 128, 256]), dtype=rng.choice(["bf16", "f32"]),
                     grad=rng.random() < 0.6, skew=rng.random() < 0.5)
            if rng.random() < 0.6:
                c["width"] = (c["width"] + 7) // 8 * 8
            if c["tokens"] * c["top_k"] * c["width"] * SIZE[c["dtype"]] > 16384 * 2 * 4096 * 2:
                continue
            if c["experts"] * c["pad"] * c["width"] > 1 << 26:
                continue
        elif op == "quant":
            transposed = rng.random() < 0.4
            dtype = rng.choice(["bf16", "f32"])
            c = dict(op=op, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 16, 16384), dtype=dtype,
                     transposed=transposed, act="relu2" if dtype == "bf16" and rng.random() < 0.3 else "none")
            if rng.random() < 0.5:
                c["cols"] = (c["cols"] + 31) // 32 * 32
            if c["rows"] * c["cols"] * SIZE[dtype] > 1 << 29:
                continue
        elif op == "product":
            train = rng.random() < 0.4
            c = dict(op=op, m=_log_int(rng, 1, 8192), n=_log_int(rng, 64, 16384), k=_log_int(rng, 64, 16384),
                     out=rng.choice(["bf16", "f32"]), train=train)
            if rng.random() < 0.5:
                c["n"], c["k"] = (c["n"] + 31) // 32 * 32, (c["k"] + 31) // 32 * 32
            if c["m"] * c["n"] * c["k"] > 8192 * 16384 * 4096:
                continue
        else:
            experts = _log_int(rng, 2, 128)
            train = rng.random() < 0.4
            c = dict(op=op, tokens=_log_int(rng, 1, 8192), width=_log_int(rng, 64, 4096),
                     out_width=_log_int(rng, 64, 8192), experts=experts, top_k=rng.randint(1, min(6, experts)),
                     pad=256 if train else rng.choice([128, 256]), train=train, skew=rng.random() < 0.5)
            if rng.random() < 0.5:
                c["width"], c["out_width"] = (c["width"] + 31) // 32 * 32, (c["out_width"] + 31) // 32 * 32
            rows = c["tokens"] * c["top_k"] + experts * c["pad"]
            if rows * c["width"] * c["out_width"] > 16384 * 2048 * 8192 or experts * c["width"] * c["out_width"] > 1 << 28:
                continue
        return c


# ------------------------------------------------------------------ the inputs

def _normal(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _rows_bound(tokens, top_k, experts, pad):
    """Rows that the sorted order can take at most: every expert's segment is a multiple of pad."""
    n = tokens * top_k
    return (n + min(experts, n) * (pad - 1) + pad - 1) // pad * pad


def _routing(case, seed):
    """Expert ids [tokens, top_k], distinct for a token; with "skew" some experts
    are chosen far more often, some slots choose nothing (-1) and a few tokens
    name an expert twice."""
    rng = np.random.default_rng(seed)
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    score = rng.gumbel(size=(T, E))
    if case["skew"]:
        score = score - 1.2 * np.log1p(rng.permutation(E))[None, :]
    idx = np.argsort(-score, axis=1)[:, :k].astype(np.int32)
    if case["skew"]:
        idx[rng.random((T, k)) < 0.02] = -1
        if k > 1:
            twice = rng.random(T) < 0.01
            idx[twice, 1] = idx[twice, 0]
    return torch.from_numpy(np.ascontiguousarray(idx)).cuda()


def _pack(v):
    """Codes and tiled scales of MXFP4 for a matrix [..., rows, cols], as a program
    that loads quantised weights has them.  Codes: two values a byte (the even column
    in the low half), rows padded to whole blocks.  Scales: one byte a block (the
    exponent plus 127), in tiles of 128 rows x 4 blocks; in a tile the byte of row r,
    block b is r % 32 * 16 + r / 32 * 4 + b; tiles along a row first, an even number."""
    *lead, rows, cols = v.shape
    v = v.reshape(-1, rows, cols).float()
    batch = v.shape[0]
    nb = (cols + BLOCK - 1) // BLOCK
    codes = torch.empty(batch, rows, nb * 16, dtype=torch.uint8, device=v.device)
    rb, cg = (rows + 127) // 128, (cols + 255) // 256 * 2
    scales = torch.zeros(batch, rb * 128, cg * 4, dtype=torch.uint8, device=v.device)
    for i in range(batch):
        q, e = _round_blocks(v[i])
        a = torch.bucketize(q.abs(), torch.tensor(E2M1, device=v.device) - 0.125) - 1
        c = (a + 8 * torch.signbit(q)).to(torch.uint8).reshape(rows, nb * 16, 2)
        codes[i] = c[..., 0] | (c[..., 1] << 4)
        scales[i, :rows, :nb] = (e + 127).to(torch.uint8)
    tiled = scales.reshape(batch, rb, 4, 32, cg, 4).permute(0, 1, 4, 3, 2, 5).contiguous()
    return codes.reshape(*lead, rows, nb * 16), tiled.reshape(*lead, rb * cg * 512)


def _routed_state(case, seed, gen):
    R = _rows_bound(case["tokens"], case["top_k"], case["experts"], case["pad"])
    return dict(idx=_routing(case, seed), R=R)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "dispatch":
        st.update(_routed_state(case, seed, gen))
        T, d, k, dt = case["tokens"], case["width"], case["top_k"], TORCH[case["dtype"]]
        st["x"] = _normal(gen, (T, d), 1.0, dt)
        st["weights"] = torch.rand((T, k), generator=gen, device="cuda") * 0.9 + 0.1
        st["out_rows"] = _normal(gen, (st["R"], d), 1.0, dt)      # the experts' outputs, in sorted order
        if case["grad"]:
            st["dy"] = _normal(gen, (T, d), 1e-2, dt)
            st["d_rows"] = _normal(gen, (st["R"], d), 1e-2, dt)   # the gradient that comes back from the experts
    elif op == "quant":
        shape = (case["cols"], case["rows"]) if case["transposed"] else (case["rows"], case["cols"])
        st["x"] = _normal(gen, shape, 1.0, TORCH[case["dtype"]])
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        w = _normal(gen, (n, k), k ** -0.5, torch.bfloat16)
        st["x"] = _normal(gen, (m, k), 1.0, torch.bfloat16)
        st["w"] = _pack(w)
        if case["train"]:
            st["wt"] = _pack(w.t())
            st["dy"] = _normal(gen, (m, n), 1e-2, torch.bfloat16)
    else:
        st.update(_routed_state(case, seed, gen))
        T, d, n, E = case["tokens"], case["width"], case["out_width"], case["experts"]
        w = _normal(gen, (E, n, d), d ** -0.5, torch.bfloat16)
        st["x"] = _normal(gen, (T, d), 1.0, torch.bfloat16)
        st["w"] = _pack(w)
        if case["train"]:
            st["wt"] = _pack(w.transpose(1, 2))
            st["d_rows"] = _normal(gen, (st["R"], n), 1e-2, torch.bfloat16)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """The buffers that a program keeps for its calls."""
    import mlp_block_backprop_gb300 as mb
    case, op = st["case"], st["case"]["op"]
    dev = dict(device="cuda")
    code = {"bf16": mb.MLPBLK_BF16, "f32": mb.MLPBLK_FP32}
    if op in ("dispatch", "experts"):
        st["sort"] = mb.MoeSort(case["tokens"], case["width"], case["experts"], case["top_k"], case["pad"],
                                dtype=case.get("dtype", "bf16"))
    if op == "dispatch":
        st["rows"] = torch.zeros_like(st["out_rows"])
        st["y"] = torch.empty_like(st["x"])
        if case["grad"]:
            st["d_out_rows"] = torch.zeros_like(st["out_rows"])
            st["d_weights"] = torch.empty_like(st["weights"])
            st["dx"] = torch.empty_like(st["x"])
    elif op == "quant":
        st["q"] = mb.Fp4Matrix(case["rows"], case["cols"])
        st["y"] = torch.empty(case["rows"], case["cols"], dtype=TORCH[case["dtype"]], **dev)
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        out = TORCH[case["out"]]
        st["xq"] = mb.Fp4Matrix(m, k)
        st["wq"] = mb.Fp4Matrix(n, k, codes=st["w"][0], scales=st["w"][1])
        st["y"] = torch.empty(m, n, dtype=out, **dev)
        if case["train"]:
            st["wtq"] = mb.Fp4Matrix(k, n, codes=st["wt"][0], scales=st["wt"][1])
            st["dyq"], st["dytq"], st["xtq"] = mb.Fp4Matrix(m, n), mb.Fp4Matrix(n, m), mb.Fp4Matrix(k, m)
            st["dx"] = torch.empty(m, k, dtype=out, **dev)
            st["dw"] = torch.empty(n, k, dtype=torch.float32, **dev)
    else:
        d, n, E, R = case["width"], case["out_width"], case["experts"], st["R"]
        st["xq"] = mb.Fp4Matrix(R, d)
        st["wq"] = mb.Fp4Matrix(n, d, batch=E, codes=st["w"][0], scales=st["w"][1])
        st["rows"] = torch.zeros(R, n, dtype=torch.bfloat16, **dev)
        if case["train"]:
            st["wtq"] = mb.Fp4Matrix(d, n, batch=E, codes=st["wt"][0], scales=st["wt"][1])
            st["dq"], st["dtq"], st["xtq"] = mb.Fp4Matrix(R, n), mb.Fp4Matrix(n, R), mb.Fp4Matrix(d, R)
            st["dx_rows"] = torch.zeros(R, d, dtype=torch.bfloat16, **dev)
            st["dw"] = torch.empty(E, n, d, dtype=torch.float32, **dev)


# -------------------------------------------------------- the framework's calls

def _run_own(st):
    case, op = st["case"], st["case"]["op"]
    if op == "dispatch":
        s = st["sort"]
        s.sort(st["idx"])
        s.permute(st["x"], st["rows"])
        s.unpermute(st["out_rows"], st["y"], weights=st["weights"], residual=st["x"])
        out = [s.count, s.seg, s.pos, s.row_map, st["rows"], st["y"]]
        if case["grad"]:
            s.unpermute_backward(st["dy"], st["out_rows"], st["weights"], st["d_out_rows"], st["d_weights"])
            s.permute_backward(st["d_rows"], st["dx"])
            out += [st["d_out_rows"], st["d_weights"], st["dx"]]
        return out
    if op == "quant":
        st["q"].quantize(st["x"], transposed=case["transposed"], act=case["act"])
        st["q"].dequantize(st["y"])
        return st["y"]
    if op == "product":
        st["xq"].quantize(st["x"])
        st["xq"].matmul(st["wq"], st["y"])
        if not case["train"]:
            return st["y"]
        st["dyq"].quantize(st["dy"])
        st["dyq"].matmul(st["wtq"], st["dx"])
        st["dytq"].quantize(st["dy"], transposed=True)
        st["xtq"].quantize(st["x"], transposed=True)
        st["dytq"].matmul(st["xtq"], st["dw"])
        return [st["y"], st["dx"], st["dw"]]
    s = st["sort"]
    s.sort(st["idx"])
    st["xq"].quantize(st["x"], sort=s, gather=True)
    st["xq"].matmul_grouped(st["wq"], s, st["rows"])
    if not case["train"]:
        return [s.count, st["rows"]]
    st["dq"].quantize(st["d_rows"], sort=s)
    st["dq"].matmul_grouped(st["wtq"], s, st["dx_rows"])
    st["dtq"].quantize(st["d_rows"], sort=s, transposed=True)
    st["xtq"].quantize(st["x"], sort=s, gather=True, transposed=True)
    st["dtq"].wgrad_grouped(st["xtq"], s, st["dw"])
    return [s.count, st["rows"], st["dx_rows"], st["dw"]]


# ---------------------------------------------------------------- the plain form

def _pow2(e):
    """2^e in float32, exactly, for integers -127 <= e <= 127."""
    return torch.tensor([2.0 ** i for i in range(-127, 128)], device=e.device)[e + 127]


def _round_blocks(v):
    """A float32 matrix in MXFP4: the elements before scaling (a multiple of 0.5,
    |.| <= 6; columns padded to whole blocks) and the blocks' exponents."""
    rows, cols = v.shape
    nb = (cols + BLOCK - 1) // BLOCK
    if nb * BLOCK != cols:
        v = torch.nn.functional.pad(v, (0, nb * BLOCK - cols))
    v = v.reshape(rows, nb, BLOCK)
    amax = v.abs().amax(dim=2)
    e = torch.frexp(amax).exponent - 3          # floor(log2(amax)) - 2
    e = torch.where(amax > 0, e, -127).clamp(min=-127)
    v = v * _pow2(-e)[..., None]
    a = v.abs()
    i = (a > 0.25).to(torch.uint8)
    for edge, even_above in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        i += (a >= edge) if even_above else (a > edge)
    q = torch.tensor(E2M1, device=v.device)[i.int()]
    return torch.copysign(q, v).reshape(rows, nb * BLOCK), e


def _rounded(v):
    """The values that a float32 matrix has after rounding to MXFP4."""
    rows, cols = v.shape
    q, e = _round_blocks(v)
    return (q.reshape(rows, -1, BLOCK) * _pow2(e)[..., None]).reshape(rows, -1)[:, :cols]


def _decoded(packed, rows, cols):
    """The values of one packed matrix."""
    codes, tiled = packed
    nb = (cols + BLOCK - 1) // BLOCK
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    c = codes.int()
    v = table[torch.stack((c & 15, c >> 4), dim=-1).reshape(rows, nb, BLOCK)]
    rb, cg = (rows + 127) // 128, (cols + 255) // 256 * 2
    s = tiled.reshape(rb, cg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cg * 4)[:rows, :nb]
    return (v * _pow2(s.int() - 127)[..., None]).reshape(rows, nb * BLOCK)[:, :cols]


def _sorted_plan(idx, experts, pad, R):
    """count, seg, pos, row_map of the sorted order: entries (token, slot) of an
    expert keep their order, segments start at multiples of pad."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    live = (flat >= 0) & (flat < experts)
    key = torch.where(live, flat, experts)
    order = torch.sort(key, stable=True).indices
    count = torch.bincount(key, minlength=experts + 1)[:experts]
    padded = (count + pad - 1) // pad * pad
    seg = torch.cat((padded.new_zeros(1), padded.cumsum(0)))
    first = torch.cat((count.new_zeros(1), count.cumsum(0)))      # where each expert's entries start in `order`
    pos = flat.new_full((n,), -1)
    k = key[order]
    rows = seg[k] + torch.arange(n, device=flat.device) - first[k]
    pos[order] = torch.where(k < experts, rows, -1)
    row_map = flat.new_full((R + 1,), -1)
    row_map[torch.where(pos >= 0, pos, R)] = torch.arange(n, device=flat.device)
    row_map = row_map[:R]
    return [t.int() for t in (count, seg)] + [pos.reshape(idx.shape).int(), row_map.int()]


def _take_rows(x, row_map, div):
    """Row r = x[row_map[r] / div], zero where nothing is mapped."""
    at = torch.where(row_map >= 0, row_map, 0).long() // div
    return x[at] * (row_map >= 0)[:, None].to(x.dtype)


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "dispatch":
        dt, k = TORCH[case["dtype"]], case["top_k"]
        count, seg, pos, row_map = _sorted_plan(st["idx"], case["experts"], case["pad"], st["R"])
        rows = _take_rows(st["x"], row_map, k)
        at, live = pos.clamp(min=0).long(), (pos >= 0).float()
        y = st["x"].float()
        for j in range(k):
            y = y + (st["weights"][:, j] * live[:, j])[:, None] * st["out_rows"][at[:, j]].float()
        out = [count, seg, pos, row_map, rows, y.to(dt)]
        if case["grad"]:
            dy = st["dy"].float()
            w = torch.cat((st["weights"].reshape(-1), st["weights"].new_zeros(1)))
            token = torch.where(row_map >= 0, row_map, 0).long() // k
            d_out = dy[token] * w[torch.where(row_map >= 0, row_map, -1).long()][:, None]
            d_w = torch.stack([(dy * st["out_rows"][at[:, j]].float()).sum(1) * live[:, j] for j in range(k)], 1)
            dx = torch.zeros_like(dy)
            for j in range(k):
                dx = dx + st["d_rows"][at[:, j]].float() * live[:, j][:, None]
            out += [d_out.to(dt), d_w, dx.to(dt)]
        return out
    if op == "quant":
        v = st["x"].float()
        if case["act"] == "relu2":
            v = v.clamp(min=0) ** 2
        return _rounded(v.t().contiguous() if case["transposed"] else v).to(TORCH[case["dtype"]])
    if op == "product":
        m, n, k, out = case["m"], case["n"], case["k"], TORCH[case["out"]]
        x = st["x"].float()
        y = (_rounded(x) @ _decoded(st["w"], n, k).t()).to(out)
        if not case["train"]:
            return y
        dy = st["dy"].float()
        dx = (_rounded(dy) @ _decoded(st["wt"], k, n).t()).to(out)
        dw = _rounded(dy.t().contiguous()) @ _rounded(x.t().contiguous()).t()
        return [y, dx, dw]
    d, n, E, k = case["width"], case["out_width"], case["experts"], case["top_k"]
    count, seg, pos, row_map = _sorted_plan(st["idx"], E, case["pad"], st["R"])
    seg_h = seg.tolist()                     # a loop over the experts needs their sizes on the host
    x = _take_rows(st["x"].float(), row_map, k)
    xq = _rounded(x)
    rows = torch.zeros(st["R"], n, device=x.device)
    for e in range(E):
        if seg_h[e + 1] > seg_h[e]:
            rows[seg_h[e]:seg_h[e + 1]] = xq[seg_h[e]:seg_h[e + 1]] @ _decoded((st["w"][0][e], st["w"][1][e]), n, d).t()
    if not case["train"]:
        return [count, rows.to(torch.bfloat16)]
    dr = st["d_rows"].float() * (row_map >= 0)[:, None].float()
    dq = _rounded(dr)
    dtq, xtq = _rounded(dr.t().contiguous()), _rounded(x.t().contiguous())
    dx_rows = torch.zeros(st["R"], d, device=x.device)
    dw = torch.zeros(E, n, d, device=x.device)
    for e in range(E):
        a, b = seg_h[e], seg_h[e + 1]
        if b > a:
            dx_rows[a:b] = dq[a:b] @ _decoded((st["wt"][0][e], st["wt"][1][e]), d, n).t()
            dw[e] = dtq[:, a:b] @ xtq[:, a:b].t()
    return [count, rows.to(torch.bfloat16), dx_rows.to(torch.bfloat16), dw]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ what a pass needs

def _live_experts(case):
    """Experts that get a token, on average."""
    return case["experts"] * (1.0 - (1.0 - case["top_k"] / case["experts"]) ** case["tokens"])


def _fp4_bytes(rows, cols):
    return rows * ((cols + 31) // 32) * 17


def work(case):
    op = case["op"]
    if op == "dispatch":
        T, d, k = case["tokens"], case["width"], case["top_k"]
        row, n = d * SIZE[case["dtype"]], T * k
        b = 4 * n + 12 * n                               # ids; weights, pos, row_map
        b += T * row + n * row + n * row + T * row       # x, rows; the experts' rows, y
        f = 2.0 * n * d
        if case["grad"]:
            b += T * row + n * row + 4 * n + n * row + T * row
            f += 4.0 * n * d
        return {"bytes": float(b), "flops": f}
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": 2.0 * n * SIZE[case["dtype"]], "flops": 4.0 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        b = 2.0 * m * k + _fp4_bytes(n, k) + m * n * SIZE[case["out"]]
        if case["train"]:
            b += 2.0 * m * n + _fp4_bytes(k, n) + m * k * SIZE[case["out"]] + 4.0 * n * k
        return {"bytes": b, "flops": 2.0 * m * n * k * (3 if case["train"] else 1)}
    T, d, n, E, k = case["tokens"], case["width"], case["out_width"], case["experts"], case["top_k"]
    live = min(_live_experts(case), T * k)
    b = 4.0 * T * k + 2.0 * T * d + live * _fp4_bytes(n, d) + 2.0 * T * k * n
    if case["train"]:
        b += 2.0 * T * k * n + live * _fp4_bytes(d, n) + 2.0 * T * k * d + 4.0 * E * n * d
    return {"bytes": b, "flops": 2.0 * T * k * n * d * (3 if case["train"] else 1)}


# ------------------------------------------------- the definition, in 64 bits

def _mx64(a):
    """MXFP4 values of a float64 matrix, block by block along its rows: the shared
    scale is 2^(floor(log2 max) - 2); an element rounds to the nearest multiple of its
    binade's step (0.5, 1 or 2 scales), ties to even, and saturates at 6 scales."""
    rows, cols = a.shape
    out = torch.zeros_like(a)
    for c in range(0, cols, 8192):
        part = a[:, c:c + 8192]
        w = part.shape[1]
        wide = torch.zeros(rows, (w + 31) // 32 * 32, dtype=torch.float64, device=a.device)
        wide[:, :w] = part
        blk = wide.view(rows, -1, 32)
        top = blk.abs().max(dim=2, keepdim=True).values
        # 2^e as a double's bit pattern: exponent field e + 1023, no fraction
        e = torch.where(top > 0, torch.frexp(top).exponent - 1 - 2, -127).clamp(min=-127).long()
        scale = ((e + 1023) << 52).view(torch.float64)
        u = blk / scale
        step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0)).double()
        u = torch.round(u / step) * step            # half to even
        out[:, c:c + 8192] = (u.clamp(-6, 6) * scale).view(rows, -1)[:, :w]
    return out


def _inputs(case, seed):
    """prepare's inputs without the framework's buffers."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _unpack64(codes, tiled, rows, cols):
    """Value by value from the byte layout: row r, column c."""
    dev = codes.device
    r = torch.arange(rows, device=dev)[:, None]
    c = torch.arange(cols, device=dev)[None, :]
    byte = codes.view(-1)[r * codes.shape[-1] + c // 2].int()
    nibble = torch.where(c % 2 == 0, byte & 15, byte >> 4)
    mag, expo = (nibble & 1).double(), (nibble >> 1 & 3).double()
    val = torch.where(expo == 0, mag * 0.5, torch.where(expo == 1, 1.0, torch.where(expo == 2, 2.0, 4.0)) * (1 + mag * 0.5))
    val = torch.where(nibble >= 8, -val, val)
    b = torch.arange((cols + 31) // 32, device=dev)[None, :]
    tile = r // 128 * ((cols + 255) // 256 * 2) + b // 4
    s = tiled.view(-1)[tile * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4].long()
    return val * ((s - 127 + 1023) << 52).view(torch.float64).repeat_interleave(32, dim=1)[:, :cols]


def _plan64(idx, experts, pad, R):
    """The sorted order, written out entry by entry."""
    flat = idx.reshape(-1).cpu().numpy()
    count = np.array([(flat == e).sum() for e in range(experts)], dtype=np.int32)
    seg = np.zeros(experts + 1, dtype=np.int32)
    for e in range(experts):
        seg[e + 1] = seg[e] + -(-int(count[e]) // pad) * pad
    pos = np.full(flat.shape, -1, dtype=np.int32)
    row_map = np.full(R, -1, dtype=np.int32)
    for e in range(experts):
        entries = np.flatnonzero(flat == e)
        pos[entries] = seg[e] + np.arange(len(entries))
        row_map[seg[e]:seg[e] + len(entries)] = entries
    dev = [torch.from_numpy(a).to(idx.device) for a in (count, seg, pos.reshape(idx.shape), row_map)]
    return dev, seg


def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "quant":
        a = st["x"].double()
        if case["act"] == "relu2":
            a = torch.relu(a).square()
        return _mx64(a.T.contiguous() if case["transposed"] else a)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        x = st["x"].double()
        y = torch.matmul(_mx64(x), _unpack64(*st["w"], n, k).T)
        if not case["train"]:
            return y
        dy = st["dy"].double()
        dx = torch.matmul(_mx64(dy), _unpack64(*st["wt"], k, n).T)
        return [y, dx, torch.matmul(_mx64(dy.T.contiguous()), _mx64(x.T.contiguous()).T)]
    k, E, R = case["top_k"], case["experts"], st["R"]
    (count, seg, pos, row_map), segh = _plan64(st["idx"], E, case["pad"], R)
    used = torch.nonzero(row_map >= 0)[:, 0]
    entry = row_map[used].long()
    x = torch.zeros(R, case["width"], dtype=torch.float64, device="cuda")
    x[used] = st["x"].double()[entry // k]
    if op == "dispatch":
        w = st["weights"].double().reshape(-1)
        y = st["x"].double()
        y.index_add_(0, entry // k, st["out_rows"].double()[used] * w[entry][:, None])
        out = [count, seg, pos, row_map, x, y]
        if case["grad"]:
            dy = st["dy"].double()
            d_out = torch.zeros_like(x)
            d_out[used] = dy[entry // k] * w[entry][:, None]
            d_w = torch.zeros_like(w)
            d_w[entry] = (dy[entry // k] * st["out_rows"].double()[used]).sum(1)
            dx = torch.zeros_like(dy)
            dx.index_add_(0, entry // k, st["d_rows"].double()[used])
            out += [d_out, d_w.reshape(pos.shape), dx]
        return out
    d, n = case["width"], case["out_width"]
    rows = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    xq = _mx64(x)
    for e in range(E):
        s = slice(int(segh[e]), int(segh[e + 1]))
        if s.stop > s.start:
            rows[s] = torch.matmul(xq[s], _unpack64(st["w"][0][e], st["w"][1][e], n, d).T)
    if not case["train"]:
        return [count, rows]
    g = torch.zeros(R, n, dtype=torch.float64, device="cuda")
    g[used] = st["d_rows"].double()[used]
    gq, gt, xt = _mx64(g), _mx64(g.T.contiguous()), _mx64(x.T.contiguous())
    dx_rows = torch.zeros(R, d, dtype=torch.float64, device="cuda")
    dw = torch.zeros(E, n, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        s = slice(int(segh[e]), int(segh[e + 1]))
        if s.stop > s.start:
            dx_rows[s] = torch.matmul(gq[s], _unpack64(st["wt"][0][e], st["wt"][1][e], d, n).T)
            dw[e] = torch.matmul(gt[:, s], xt[:, s].T)
    return [count, rows, dx_rows, dw]
