"""The work of the routing, norm and orthogonalising operators, as cases that can be timed.

They stand around the routed experts of a training or serving step:

  route  a token's logits -> the experts that it goes to and their weights: softmax or
         sigmoid scores, a bias for balance that only selects, groups of experts, top-k,
         renormalised weights; a training pass adds the gradient of the logits
  norm   the residual stream's sum, its RMSNorm, and the result as E4M3 codes with a
         float32 scale for each row (or each 128 values of a row); a training pass adds
         the gradients of the summands and of gamma
  ortho  a weight's momentum -> the nearest orthogonal matrix, roughly: five Newton-Schulz
         steps X <- a X + (b G + c G^2) X, G = X X^T, from X = U / |U|, as Muon takes them

With ``own`` false, ``run`` computes a case in plain torch operations; with ``own`` true it
calls mlp_block_backprop_gb300.
"""

import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E4M3_MAX = 448.0
STEPS, NS = 5, (3.4445, -4.7750, 2.0315)     # Newton-Schulz steps and coefficients
TINY = 1e-20                                 # added to the sum that renormalises
EPS = 1e-6                                   # of the norm
ORTHO_EPS = 1e-7                             # added to |U|


def listed():
    return [
        # a serving step of 8 sequences through many experts in groups: latency alone
        dict(name="route_decode", op="route", tokens=8, experts=256, top_k=8, score="sigmoid", groups=8, top_groups=4,
             bias=True, renorm=True, dtype="f32", grad=False, masked=False),
        # a training microbatch over a few experts, plain softmax weights
        dict(name="route_few", op="route", tokens=8192, experts=8, top_k=2, score="softmax", groups=1, top_groups=1,
             bias=False, renorm=False, dtype="bf16", grad=True, masked=False),
        # an odd number of tokens, some of them padding, and an odd number of experts, some closed to some tokens
        dict(name="route_ragged", op="route", tokens=4097, experts=60, top_k=6, score="softmax", groups=1, top_groups=1,
             bias=True, renorm=True, dtype="f32", grad=True, masked=True),
        # a training batch over many experts in groups, balanced by a bias
        dict(name="route_many", op="route", tokens=65536, experts=256, top_k=8, score="sigmoid", groups=8, top_groups=4,
             bias=True, renorm=True, dtype="bf16", grad=True, masked=False),
        # the rows of 8 sequences between two layers of a serving step
        dict(name="norm_token", op="norm", tokens=8, width=4096, dtype="bf16", block=0, residual=True, grad=False),
        # odd sizes in float32, no residual branch
        dict(name="norm_odd", op="norm", tokens=4097, width=1001, dtype="f32", block=0, residual=False, grad=True),
        # a long prompt of wide rows, a scale for each 128 values
        dict(name="norm_prompt", op="norm", tokens=8192, width=8192, dtype="bf16", block=128, residual=True, grad=False),
        # a training microbatch of the large block's width, forward and backward
        dict(name="norm_train", op="norm", tokens=16384, width=4096, dtype="bf16", block=0, residual=True, grad=True),
        # a small projection: latency of the dependent products
        dict(name="ortho_small", op="ortho", batch=1, rows=256, cols=256, dtype="f32"),
        # odd sizes, taller than wide, bf16 momentum
        dict(name="ortho_odd", op="ortho", batch=3, rows=1000, cols=333, dtype="bf16"),
        # the up projections of eight routed experts
        dict(name="ortho_experts", op="ortho", batch=8, rows=1024, cols=2048, dtype="f32"),
        # the large block's up projection
        dict(name="ortho_large", op="ortho", batch=1, rows=16384, cols=4096, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above."""
    while True:
        op = rng.choice(["route", "norm", "ortho"])
        if op == "route":
            groups = rng.choice([1, 1, 2, 4, 8])
            per = _log_int(rng, 4, 256 // groups)
            top_groups = rng.randint(1, groups)
            c = dict(op=op, tokens=_log_int(rng, 1, 65536), experts=groups * per,
                     top_k=rng.randint(1, min(16, top_groups * per)), score=rng.choice(["softmax", "sigmoid"]),
                     groups=groups, top_groups=top_groups, bias=rng.random() < 0.5, renorm=rng.random() < 0.6,
                     dtype=rng.choice(["bf16", "f32"]), grad=rng.random() < 0.6, masked=rng.random() < 0.3)
            if c["tokens"] * c["experts"] * SIZE[c["dtype"]] > 65536 * 256 * 2:
                continue
        elif op == "norm":
            c = dict(op=op, tokens=_log_int(rng, 1, 65536), width=_log_int(rng, 32, 16384), dtype=rng.choice(["bf16", "f32"]),
                     block=rng.choice([0, 128]), residual=rng.random() < 0.7, grad=rng.random() < 0.5)
            if rng.random() < 0.6:
                c["width"] = (c["width"] + 7) // 8 * 8
            if c["tokens"] * c["width"] * SIZE[c["dtype"]] > 16384 * 4096 * 2:
                continue
        else:
            c = dict(op=op, batch=_log_int(rng, 1, 16), rows=_log_int(rng, 32, 16384), cols=_log_int(rng, 32, 16384),
                     dtype=rng.choice(["bf16", "f32"]))
            if rng.random() < 0.5:
                c["rows"], c["cols"] = (c["rows"] + 31) // 32 * 32, (c["cols"] + 31) // 32 * 32
            m, n = sorted((c["rows"], c["cols"]))
            if c["batch"] * m * m * (3 * n + m) > 4096 * 4096 * 2 * (3 * 4096 + 2048) or c["batch"] * m * n > 1 << 26:
                continue
        return c


# ------------------------------------------------------------------ the inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        logits = _normal(gen, (T, E), 1.5) + _normal(gen, (E,), 0.5)     # some experts are liked by every token
        if case["masked"]:
            closed = torch.rand((T, E), generator=gen, device="cuda") < 0.2
            padding = torch.rand((T, 1), generator=gen, device="cuda") < 0.1
            logits = torch.where(closed | padding, -math.inf, logits)
        st["logits"] = logits.to(TORCH[case["dtype"]])
        st["bias"] = _normal(gen, (E,), 0.05) if case["bias"] else None
        if case["grad"]:
            st["d_weights"] = _normal(gen, (T, k), 1e-2)
    elif op == "norm":
        T, d, dt = case["tokens"], case["width"], TORCH[case["dtype"]]
        channel = 1.0 + 4.0 * (torch.rand(d, generator=gen, device="cuda") < 0.01).float()   # a few loud channels
        st["x"] = (_normal(gen, (T, d)) * channel).to(dt)
        st["residual"] = _normal(gen, (T, d), 0.5).to(dt) if case["residual"] else None
        st["gamma"] = (1.0 + _normal(gen, (d,), 0.02)).to(dt)
        if case["grad"]:
            st["dn"] = _normal(gen, (T, d), 1e-2).to(dt)
            st["d_sum"] = _normal(gen, (T, d), 1e-2).to(dt)
    else:
        # momentum: a few strong directions over noise
        b, r, c = case["batch"], case["rows"], case["cols"]
        rank = min(16, r, c)
        strong = 4.0 / torch.arange(1, rank + 1, device="cuda", dtype=torch.float32)
        u = _normal(gen, (b, r, c), 1e-3)
        lead = (_normal(gen, (b, r, rank)) * strong) @ _normal(gen, (b, rank, c))
        st["u"] = (u + 1e-3 * (r ** -0.5 + c ** -0.5) * lead).to(TORCH[case["dtype"]])
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """The handles and buffers that a program keeps for its calls."""
    import mlp_block_backprop_gb300 as mb
    case, op = st["case"], st["case"]["op"]
    dev = dict(device="cuda")
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        st["router"] = mb.MoeRouter(T, E, k, score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                                    renorm=case["renorm"], dtype=case["dtype"])
        st["ids"] = torch.empty(T, k, dtype=torch.int32, **dev)
        st["weights"] = torch.empty(T, k, dtype=torch.float32, **dev)
        if case["grad"]:
            st["d_logits"] = torch.empty_like(st["logits"])
    elif op == "norm":
        T, d = case["tokens"], case["width"]
        st["norm"] = mb.AddRmsNorm(T, d, eps=EPS, dtype=case["dtype"], block=case["block"])
        st["sum"] = torch.empty_like(st["x"]) if case["residual"] else st["x"]
        st["codes"] = torch.empty(T, d, dtype=torch.float8_e4m3fn, **dev)
        st["scales"] = torch.empty(T, (d + 127) // 128 if case["block"] else 1, dtype=torch.float32, **dev)
        if case["grad"]:
            st["dx"] = torch.empty_like(st["x"])
            st["dgamma"] = torch.empty(d, dtype=torch.float32, **dev)
    else:
        b, r, c = case["batch"], case["rows"], case["cols"]
        st["ortho"] = mb.Orthogonalizer(r, c, batch=b, steps=STEPS, coefficients=NS, eps=ORTHO_EPS, dtype=case["dtype"])
        st["o"] = torch.empty(b, r, c, dtype=torch.bfloat16, **dev)


# -------------------------------------------------------- the framework's calls

def _run_own(st):
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        st["router"].route(st["logits"], st["ids"], st["weights"], bias=st["bias"])
        if not case["grad"]:
            return [st["ids"], st["weights"]]
        st["router"].route_backward(st["logits"], st["ids"], st["d_weights"], st["d_logits"])
        return [st["ids"], st["weights"], st["d_logits"]]
    if op == "norm":
        n = st["norm"]
        n.forward(st["x"], st["gamma"], codes=st["codes"], scales=st["scales"], residual=st["residual"],
                  sum=st["sum"] if case["residual"] else None)
        out = [st["codes"], st["scales"], n.rstd] + ([st["sum"]] if case["residual"] else [])
        if case["grad"]:
            n.backward(st["dn"], st["sum"], st["gamma"], st["dx"], st["dgamma"], d_sum=st["d_sum"], overwrite=True)
            out += [st["dx"], st["dgamma"]]
        return out
    st["ortho"].orthogonalize(st["u"], st["o"])
    return st["o"]


# ---------------------------------------------------------------- the plain form

def _scores(logits, score):
    """Scores in 64 bits (their order decides what is selected), 0 for closed experts."""
    v = logits.double()
    live = v > -math.inf
    if score == "sigmoid":
        return torch.where(live, 1.0 / (1.0 + torch.exp(-v)), 0.0), live
    top = v.amax(dim=1, keepdim=True)
    e = torch.exp(v - torch.where(top > -math.inf, top, 0.0))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300), live


def _route(st):
    case = st["case"]
    T, E, k, G = case["tokens"], case["experts"], case["top_k"], case["groups"]
    s, live = _scores(st["logits"], case["score"])
    key = s if st["bias"] is None else s + st["bias"].double()
    key = torch.where(live, key, -math.inf)
    if case["top_groups"] < G:
        best = key.reshape(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        mark = best[:, :, 0] + torch.where(best > -math.inf, best, 0.0)[:, :, 1:].sum(dim=2)   # the two best keys' sum
        kept = mark.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter(1, kept, True)
        key = torch.where(open_.repeat_interleave(E // G, dim=1), key, -math.inf)
    found, ids = key.sort(dim=1, descending=True, stable=True)
    found, ids = found[:, :k] > -math.inf, ids[:, :k]
    picked = torch.where(found, s.gather(1, ids), 0.0)
    total = picked.sum(dim=1, keepdim=True) + TINY if case["renorm"] else torch.ones_like(picked[:, :1])
    return s, ids, found, picked, total


def _run_route(st):
    case = st["case"]
    s, ids, found, picked, total = _route(st)
    weights = picked / total
    out = [torch.where(found, ids, -1).int(), weights.float()]
    if case["grad"]:
        g = torch.where(found, st["d_weights"].double(), 0.0)
        if case["renorm"]:
            g = (g - (g * weights).sum(dim=1, keepdim=True)) / total
        ds = torch.zeros_like(s).scatter(1, ids, torch.where(found, g, 0.0))
        if case["score"] == "sigmoid":
            dl = ds * s * (1.0 - s)
        else:
            dl = s * (ds - (ds * s).sum(dim=1, keepdim=True))
        out.append(dl.to(st["logits"].dtype))
    return out


def _run_norm(st):
    case, dt = st["case"], TORCH[st["case"]["dtype"]]
    T, d, block = case["tokens"], case["width"], case["block"]
    x = st["x"]
    s = x if st["residual"] is None else (x.float() + st["residual"].float()).to(dt)
    v = s.double()                                   # codes next to a border need more than 32 bits
    rstd = 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    n = v * rstd * st["gamma"].double()
    parts = (d + 127) // 128 if block else 1
    a = n.abs()
    if block:
        a = torch.nn.functional.pad(a, (0, parts * 128 - d)).reshape(T, parts, 128).amax(dim=2)
    else:
        a = a.amax(dim=1, keepdim=True)
    scales = torch.where(a > 0, a / E4M3_MAX, 1.0).float()
    wide = scales.double().repeat_interleave(128, dim=1)[:, :d] if block else scales.double()
    codes = (n / wide).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    out = [codes, scales, rstd[:, 0].float()] + ([s] if st["residual"] is not None else [])
    if case["grad"]:
        dn = st["dn"].double()                       # dgamma sums over every token
        xh = v * rstd
        g = dn * st["gamma"].double()
        dx = st["d_sum"].double() + rstd * (g - xh * (g * xh).mean(dim=1, keepdim=True))
        out += [dx.to(dt), (dn * xh).sum(dim=0).float()]
    return out


def _run_ortho(st):
    a, b, c = NS
    x = st["u"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + ORTHO_EPS)
    for _ in range(STEPS):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


def run(state):
    if own:
        return _run_own(state)
    return {"route": _run_route, "norm": _run_norm, "ortho": _run_ortho}[state["case"]["op"]](state)


# ------------------------------------------------------------ what a pass needs

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        b = T * E * SIZE[case["dtype"]] + 8.0 * T * k
        f = 10.0 * T * E
        if case["grad"]:
            b += T * E * SIZE[case["dtype"]] + 4.0 * T * k
            f += 6.0 * T * k
        return {"bytes": float(b), "flops": f}
    if op == "norm":
        n = case["tokens"] * case["width"]
        row = SIZE[case["dtype"]]
        b = n * (row + (2 * row if case["residual"] else 0) + 1)
        f = 8.0 * n
        if case["grad"]:
            b += 3 * n * row + 4 * case["width"]     # dn, d_sum, dx
            f += 10.0 * n
        return {"bytes": float(b), "flops": f}
    m, n = sorted((case["rows"], case["cols"]))
    size = case["batch"] * m * n
    # G and G^2 are symmetric: half of their products
    return {"bytes": float(size * (SIZE[case["dtype"]] + 2)), "flops": STEPS * case["batch"] * float(m) * m * (3.0 * n + m)}


# ------------------------------------------------- the definition, in 64 bits

def _inputs(case, seed):
    """prepare's inputs without the framework's buffers."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_route(st, case):
    """The definition by comparisons: an expert's place is the number of experts that come before it."""
    T, E, k, G = case["tokens"], case["experts"], case["top_k"], case["groups"]
    l = st["logits"].double()
    bias = torch.zeros(E, dtype=torch.float64, device=l.device) if st["bias"] is None else st["bias"].double()
    ids, weights, grads = [], [], []
    for at in range(0, T, 1024):
        v = l[at:at + 1024]
        t = v.shape[0]
        shut = torch.isneginf(v)
        if case["score"] == "sigmoid":
            p = torch.sigmoid(v)
        else:
            p = torch.nan_to_num(torch.softmax(v, dim=1), nan=0.0)
        key = (p + bias).masked_fill(shut, -math.inf)
        i = torch.arange(E, device=l.device)

        def place(q):
            """How many come before each: a larger value, or the same with a lower index."""
            j = torch.arange(q.shape[1], device=q.device)
            return ((q[:, None, :] > q[:, :, None]) | ((q[:, None, :] == q[:, :, None]) & (j[None, :] < j[:, None]))).sum(2)

        if case["top_groups"] < G:
            parts = key.view(t, G, E // G)
            first = parts.max(dim=2)
            rest = parts.scatter(2, first.indices[:, :, None], -math.inf).amax(dim=2)
            mark = first.values + rest.masked_fill(torch.isneginf(rest), 0.0)
            shut_group = place(mark) >= case["top_groups"]
            key = key.masked_fill(shut_group[:, i // (E // G)], -math.inf)
        order = place(key)
        chosen = (order < k) & ~torch.isneginf(key)
        slot = torch.full((t, k + 1), -1, dtype=torch.int32, device=l.device)
        slot.scatter_(1, torch.where(chosen, order, k), i.int().expand(t, E))
        slot = slot[:, :k]
        taken = p * chosen
        total = taken.sum(1, keepdim=True) + TINY if case["renorm"] else 1.0
        at_slot = slot.clamp(min=0).long()
        w = (taken / total).gather(1, at_slot) * (slot >= 0)
        ids.append(slot)
        weights.append(w)
        if case["grad"]:
            g = st["d_weights"][at:at + 1024].double() * (slot >= 0)
            dense = torch.zeros_like(p).scatter_add_(1, at_slot, g)
            if case["renorm"]:
                dense = (dense - (g * w).sum(1, keepdim=True)) / total * chosen
            if case["score"] == "sigmoid":
                grads.append(dense * p * torch.sigmoid(-v))
            else:
                grads.append(p * dense - p * (p * dense).sum(1, keepdim=True))
    return [torch.cat(x) for x in ([ids, weights, grads] if case["grad"] else [ids, weights])]


def _e4m3(v):
    """Nearest E4M3 value, ties to even: multiples of 2^(e-3) in [2^e, 2^(e+1)), of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(st, case):
    T, d = case["tokens"], case["width"]
    x = st["x"].double()
    if st["residual"] is not None:
        # the sum is kept, and normed, in the stream's own type
        x = (x + st["residual"].double()).to(TORCH[case["dtype"]]).double()
    r = torch.rsqrt(x.pow(2).sum(1) / d + EPS)
    n = x * r[:, None] * st["gamma"].double()[None, :]
    if case["block"]:
        scales = torch.stack([n[:, c:c + 128].abs().max(dim=1).values for c in range(0, d, 128)], dim=1) / E4M3_MAX
    else:
        scales = n.abs().max(dim=1, keepdim=True).values / E4M3_MAX
    scales = torch.where(scales == 0, 1.0, scales)
    held = scales.float().double()                # codes go by the scale as it is held
    column = torch.arange(d, device=n.device) // 128 if case["block"] else torch.zeros(d, dtype=torch.long, device=n.device)
    out = [_e4m3(n / held[:, column]), scales, r]
    if st["residual"] is not None:
        out.append(x)
    if case["grad"]:
        dn, gamma = st["dn"].double(), st["gamma"].double()
        dot = (dn * gamma * x).sum(1) / d
        out.append(st["d_sum"].double() + dn * gamma * r[:, None] - x * (r.pow(3) * dot)[:, None])
        out.append(torch.einsum("td,td,t->d", dn, x, r))
    return out


def exact(case, seed):
    if case["op"] == "ortho" and case["batch"] * min(case["rows"], case["cols"]) ** 2 * max(case["rows"], case["cols"]) > 1 << 39:
        return None
    st = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(st, case)
    if case["op"] == "norm":
        return _exact_norm(st, case)
    a, b, c = NS
    out = []
    for u in st["u"].double():
        v = u / (torch.linalg.vector_norm(u) + ORTHO_EPS)
        for _ in range(STEPS):
            # the odd polynomial of the singular values, by products on the short side
            if v.shape[0] > v.shape[1]:
                g = v.T @ v
                v = a * v + b * (v @ g) + c * (v @ g @ g)
            else:
                g = v @ v.T
                v = a * v + b * (g @ v) + c * (g @ (g @ v))
        out.append(v)
    return torch.stack(out)
