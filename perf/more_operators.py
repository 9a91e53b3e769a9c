"""Measured cases of the mixture-of-experts operators and of the projection with an
epilogue, on Q2_K weights (84 bytes per 256 weights).

``linear``     y = act(x W^T + bias) + residual; ``save`` also returns z = x W^T +
               bias, which the backward pass reads.
``linear_bwd`` its backward pass with the weights frozen: dz, dx and dbias.
``sort``       tokens to their experts: where each (token, slot) lands in expert
               order, and the rows of x in that order; ``back`` also takes the
               gradient of x from that of the sorted rows.
``combine``    the experts' rows back to their tokens, with the router's weights
               and a residual.
``combine_bwd`` its gradients: of the experts' rows and of the router's weights.
``experts``    products of sorted rows with their own experts' matrices: the gated
               block or a projection, forward or backward (``kind``).

``run`` computes them in elementary torch operations in 32 bits (``own`` false),
or by the calls that a user of the package makes (``own`` true).
"""

import math

import torch

own = False

QK, BLOCK = 256, 84
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
# the most work of a drawn case: multiply-adds, and elements of sorted rows
MOST_PRODUCTS = 512 * 14336 * 4096
MOST_EXPERT_WEIGHTS = 64 * 2048 * 7168
MOST_ROWS = 1024 * 8 * 7168


def listed():
    linear = {"op": "linear", "act": "none", "bias": False, "residual": False, "save": False}
    return [
        # a handful of tokens through the tiny workload's matrix: nothing but latency
        dict(linear, name="linear tiny m4", dtype="f32", m=4, n=8, k=256, act="gelu", bias=True),
        # decode: one token's FFN down projection, added to the residual stream
        dict(linear, name="linear decode m1", dtype="f32", m=1, n=4096, k=14336, residual=True),
        # a short prompt through a matrix of odd sizes (rows that start off 16 bytes)
        dict(linear, name="linear ragged m77", dtype="bf16", m=77, n=4999, k=2816, act="silu",
             bias=True, residual=True),
        # a training micro-batch through the first half of a plain block
        dict(linear, name="linear train m512", dtype="bf16", m=512, n=7168, k=7168, act="gelu",
             bias=True, save=True),
        # its backward pass, at the FFN's width
        {"name": "linear bwd m512", "op": "linear_bwd", "dtype": "bf16", "m": 512, "n": 14336,
         "k": 4096, "act": "gelu", "bias": True},
        # one token to 8 of 64 experts: a decode step of the routed layer
        {"name": "sort decode m1", "op": "sort", "dtype": "f32", "m": 1, "top_k": 8, "experts": 64,
         "k": 7168, "pad": 0.0, "back": False},
        # a micro-batch to its experts, and the gradient on its way back
        {"name": "sort train m512", "op": "sort", "dtype": "bf16", "m": 512, "top_k": 8,
         "experts": 64, "k": 7168, "pad": 0.0, "back": True},
        # the same layer's outputs back to their tokens, onto the residual stream
        {"name": "combine m512", "op": "combine", "dtype": "bf16", "m": 512, "top_k": 8,
         "experts": 64, "n": 7168, "pad": 0.0, "weights": True, "residual": True},
        # gradients of a padded batch
        {"name": "combine bwd m1024", "op": "combine_bwd", "dtype": "bf16", "m": 1024, "top_k": 8,
         "experts": 64, "n": 7168, "pad": 0.1},
        # decode: one token's eight experts, gate and up
        {"name": "experts decode m1", "op": "experts", "kind": "gated", "dtype": "f32", "m": 1,
         "top_k": 8, "experts": 64, "n": 2048, "k": 7168, "act": "silu"},
        # prefill: 512 tokens through their experts' down projections
        {"name": "experts prefill m512", "op": "experts", "kind": "linear", "dtype": "bf16",
         "m": 512, "top_k": 8, "experts": 64, "n": 7168, "k": 2048, "act": "none"},
        # a few tokens' gradients through small experts of odd sizes
        {"name": "experts bwd ragged m75", "op": "experts", "kind": "gated_bwd", "dtype": "bf16",
         "m": 75, "top_k": 3, "experts": 10, "n": 1001, "k": 1280, "act": "gelu"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "sort", "combine", "combine_bwd", "experts",
                     "experts"])
    act = rng.choice(["none", "silu", "gelu"])
    if op in ("linear", "linear_bwd"):
        while True:
            m, n, k = _log_int(rng, 1, 2048), _log_int(rng, 8, 14336), QK * _log_int(rng, 1, 56)
            if m * n * k <= MOST_PRODUCTS:
                break
        case = {"op": op, "m": m, "n": n, "k": k, "act": act, "bias": rng.random() < 0.5}
        # 32-bit activations are the decode form; larger batches are held in bf16
        case["dtype"] = rng.choice(["f32", "bf16"]) if m <= 8 and op == "linear" else "bf16"
        if op == "linear":
            case.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        return case
    experts = _log_int(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    if op != "experts":
        while True:
            m, width = _log_int(rng, 1, 8192), _log_int(rng, 8, 14336)
            if m * top_k * width <= MOST_ROWS:
                break
        case = {"op": op, "dtype": rng.choice(["f32", "bf16"]), "m": m, "top_k": top_k,
                "experts": experts, "k" if op == "sort" else "n": width,
                "pad": rng.choice([0.0, 0.0, 0.3])}
        if case["dtype"] == "f32" and 2 * m * top_k * width > MOST_ROWS:
            case["dtype"] = "bf16"
        if op == "sort":
            case["back"] = rng.random() < 0.5
        if op == "combine":
            case.update(weights=rng.random() < 0.8, residual=rng.random() < 0.5)
        return case
    kind = rng.choice(["gated", "linear", "gated_bwd", "linear_bwd"])
    each = 2 if kind.startswith("gated") else 1
    while True:
        m, n, k = _log_int(rng, 1, 512), _log_int(rng, 8, 7168), QK * _log_int(rng, 1, 28)
        if each * experts * n * k <= MOST_EXPERT_WEIGHTS and each * m * top_k * n * k <= MOST_PRODUCTS:
            break
    if each == 2 and act == "none":
        act = "silu"
    dtype = "f32" if m == 1 and kind in ("gated", "linear") and rng.random() < 0.5 else "bf16"
    return {"op": op, "kind": kind, "dtype": dtype, "m": m, "top_k": top_k, "experts": experts,
            "n": n, "k": k, "act": act}


# ---- inputs ------------------------------------------------------------------

def _blocks(gen, n, k):
    """Random Q2_K rows whose weights have a root mean square of about 1.5 / sqrt(k),
    so that a projection of unit activations stays of order one."""
    nb = k // QK
    w = torch.randint(0, 256, (n, nb, BLOCK), dtype=torch.uint8, device="cuda", generator=gen)
    top = 0.05 * 1.5 / (0.43 * math.sqrt(k))
    d = top * (0.02 + 0.98 * torch.rand((n, nb, 2), device="cuda", generator=gen))
    w[..., 80:] = d.to(torch.float16).view(torch.uint8).view(n, nb, 4)
    return w.reshape(-1)


def _tensor(gen, dtype, *shape, scale=1.0):
    return (scale * torch.randn(shape, device="cuda", generator=gen)).to(dtype)


def _router(gen, case):
    """(ids, weights) of a router whose experts are not equally liked: each token's
    top_k distinct experts and their softmax weights; the last tokens of a padded
    batch have none (-1)."""
    m, top_k, e = case["m"], case["top_k"], case["experts"]
    liked = 0.5 * torch.randn(e, device="cuda", generator=gen)
    logits = liked + torch.randn((m, e), device="cuda", generator=gen)
    best, ids = torch.topk(logits, top_k)
    ids = ids.to(torch.int32)
    real = m - int(case.get("pad", 0.0) * m)
    ids[real:] = -1
    return ids, torch.softmax(best, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, dt = case["op"], case["m"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op in ("linear", "linear_bwd"):
        n, k = case["n"], case["k"]
        s["w"] = _blocks(gen, n, k)
        if op == "linear":
            s["x"] = _tensor(gen, dt, m, k)
            s["bias"] = _tensor(gen, torch.float32, n) if case["bias"] else None
            s["residual"] = _tensor(gen, dt, m, n) if case["residual"] else None
        else:
            s["dy"] = _tensor(gen, dt, m, n, scale=0.1)
            s["z"] = _tensor(gen, dt, m, n, scale=1.5) if case["act"] != "none" else None
        return s
    ids, weights = _router(gen, case)
    if op == "sort":
        s["ids"], s["x"] = ids, _tensor(gen, dt, m, case["k"])
        if case["back"]:
            s["dxs"] = _tensor(gen, dt, m * case["top_k"], case["k"], scale=0.1)
        return s
    s["rows"], s["order"], s["offsets"] = _route(ids, case["experts"])
    if op in ("combine", "combine_bwd"):
        n = case["n"]
        s["ys"] = _tensor(gen, dt, m * case["top_k"], n)
        s["weights"] = weights if op == "combine_bwd" or case["weights"] else None
        if op == "combine":
            s["residual"] = _tensor(gen, dt, m, n) if case["residual"] else None
        else:
            s["dy"] = _tensor(gen, dt, m, n, scale=0.1)
        return s
    # the experts' rows as the host counts them: a plan for the plain form's loop
    s["ends"] = s["offsets"].tolist()
    n, k, e, r = case["n"], case["k"], case["experts"], m * case["top_k"]
    s["w"] = _blocks(gen, e * n, k)
    if case["kind"].startswith("gated"):
        s["w2"] = _blocks(gen, e * n, k)
    if case["kind"] in ("gated", "linear"):
        s["x"] = _tensor(gen, dt, r, k)
        if case["kind"] == "linear":
            s["bias"] = _tensor(gen, torch.float32, e, n) if case["act"] != "none" else None
    else:
        s["dy"] = _tensor(gen, dt, r, n, scale=0.1)
        if case["kind"] == "gated_bwd":
            s["gate"], s["up"] = _tensor(gen, dt, r, n, scale=1.5), _tensor(gen, dt, r, n, scale=1.5)
        else:
            s["z"] = _tensor(gen, dt, r, n, scale=1.5) if case["act"] != "none" else None
    return s


# ---- plain forms ---------------------------------------------------------------

def _route(ids, experts):
    """(rows, order, offsets): where each (token, slot) lands when they are ordered by
    expert, those of one expert as they came, those without an expert last; which one
    each place holds; where each expert's places begin and the last one's end."""
    key = torch.where((ids >= 0) & (ids < experts), ids, experts).reshape(-1)
    hits = (key.view(-1, 1) == torch.arange(experts + 1, device=ids.device)).to(torch.int32)
    before = torch.cumsum(hits, 0, dtype=torch.int32)
    ends = torch.cumsum(before[-1], 0, dtype=torch.int32)
    offsets = ends - before[-1]
    rows = (offsets.gather(0, key.long())
            + before.gather(1, key.long().view(-1, 1)).view(-1) - 1)
    order = torch.empty_like(rows)
    order[rows.long()] = torch.arange(rows.numel(), device=ids.device, dtype=torch.int32)
    return rows.view(ids.shape), order, offsets


def _weights(w, n, k):
    """The rows of Q2_K blocks as 32-bit values: d (sc & 15) q - dmin (sc >> 4)."""
    b = w.view(n, k // QK, BLOCK)
    d = b[..., 80:].contiguous().view(torch.float16).to(torch.float32)
    sc = b[..., :16].view(n, -1, 2, 4, 2, 1)                       # half, shift, segment
    q = b[..., 16:80].view(n, -1, 2, 1, 2, 16)                     # half, -, segment, lane
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=w.device).view(1, 1, 1, 4, 1, 1)
    q = ((q >> shift) & 3).to(torch.float32)
    dl = d[..., 0].view(n, -1, 1, 1, 1, 1) * (sc & 15).to(torch.float32)
    ml = d[..., 1].view(n, -1, 1, 1, 1, 1) * (sc >> 4).to(torch.float32)
    return (dl * q - ml).view(n, k)


GELU_C, GELU_A = math.sqrt(2 / math.pi), 0.044715


def _act(g, act):
    if act == "none":
        return g
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(GELU_C * (g + GELU_A * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return sg * (1 + g * (1 - sg))
    t = torch.tanh(GELU_C * (g + GELU_A * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * g * g)


def _plain_linear(x, w, n, k, act, bias, residual):
    z = x.float() @ _weights(w, n, k).T
    if bias is not None:
        z = z + bias
    y = _act(z, act)
    return (y if residual is None else y + residual.float()), z


def _plain_linear_bwd(dy, z, act):
    return dy.float() if act == "none" else dy.float() * _act_slope(z.float(), act)


def _plain_experts(s):
    case = s["case"]
    n, k, dt, act, kind = case["n"], case["k"], DTYPES[case["dtype"]], case["act"], case["kind"]
    mat = n * (k // QK) * BLOCK
    back = kind.endswith("bwd")
    r = case["m"] * case["top_k"]
    wide = torch.empty((r, k if back else n), dtype=dt, device="cuda")
    if back:
        dbias = torch.zeros((case["experts"], n), device="cuda")
        if kind == "gated_bwd":
            dy, g, u = s["dy"].float(), s["gate"].float(), s["up"].float()
            d1, d2 = dy * u * _act_slope(g, act), dy * _act(g, act)
        else:
            d1 = _plain_linear_bwd(s["dy"], s["z"], act)
    for e in range(case["experts"]):
        lo, hi = s["ends"][e], s["ends"][e + 1]
        if hi == lo:
            continue
        w = _weights(s["w"][e * mat:(e + 1) * mat], n, k)
        if kind == "linear":
            z = s["x"][lo:hi].float() @ w.T
            if s["bias"] is not None:
                z = z + s["bias"][e]
            wide[lo:hi] = _act(z, act).to(dt)
            continue
        if kind == "linear_bwd":
            wide[lo:hi] = (d1[lo:hi] @ w).to(dt)
            dbias[e] = d1[lo:hi].sum(0)
            continue
        w2 = _weights(s["w2"][e * mat:(e + 1) * mat], n, k)
        if kind == "gated":
            x = s["x"][lo:hi].float()
            wide[lo:hi] = (_act(x @ w.T, act) * (x @ w2.T)).to(dt)
        else:
            wide[lo:hi] = (d1[lo:hi] @ w + d2[lo:hi] @ w2).to(dt)
    if kind == "linear":
        return {"y": wide}
    if kind == "gated":
        return {"h": wide}
    if kind == "linear_bwd":
        return {"dx": wide, "dz": d1.to(dt), "dbias": dbias}
    return {"dx": wide, "dgate": d1.to(dt), "dup": d2.to(dt)}


def _plain(s):
    case = s["case"]
    op, m, dt = case["op"], case["m"], DTYPES[case["dtype"]]
    if op == "linear":
        y, z = _plain_linear(s["x"], s["w"], case["n"], case["k"], case["act"], s["bias"],
                             s["residual"])
        return {"y": y.to(dt), "z": z.to(dt)} if case["save"] else {"y": y.to(dt)}
    if op == "linear_bwd":
        dz = _plain_linear_bwd(s["dy"], s["z"], case["act"])
        out = {"dx": (dz @ _weights(s["w"], case["n"], case["k"])).to(dt), "dz": dz.to(dt)}
        return dict(out, dbias=dz.sum(0)) if case["bias"] else out
    if op == "experts":
        return _plain_experts(s)
    top_k = case["top_k"]
    if op == "sort":
        rows, order, offsets = _route(s["ids"], case["experts"])
        real = torch.arange(m * top_k, device="cuda") < offsets[-1]
        xs = torch.where(real.view(-1, 1), s["x"][(order // top_k).long()], 0)
        out = {"xs": xs, "rows": rows, "order": order, "offsets": offsets}
        if case["back"]:
            g = torch.where((rows < offsets[-1]).unsqueeze(-1), s["dxs"][rows.long()].float(), 0)
            out["dx"] = g.sum(1).to(dt)
        return out
    rows, used = s["rows"], (s["rows"] < s["offsets"][-1]).unsqueeze(-1)
    if op == "combine":
        ys = torch.where(used, s["ys"][rows.long()].float(), 0)
        if s["weights"] is not None:
            ys = ys * s["weights"].unsqueeze(-1)
        y = ys.sum(1)
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(dt)}
    dy = s["dy"].float().unsqueeze(1)
    dweights = torch.where(used, s["ys"][rows.long()].float() * dy, 0).sum(-1)
    dys = torch.empty_like(s["ys"])
    dys[rows.view(-1).long()] = torch.where(used, s["weights"].unsqueeze(-1) * dy, 0).to(dt).view(m * top_k, -1)
    return {"dys": dys, "dweights": dweights}


def run(s):
    if not own:
        return _plain(s)
    import ggml_q2_quantized_gb300 as q2k
    case = s["case"]
    op = case["op"]
    act = None if case.get("act") == "none" else case.get("act")
    if op == "linear":
        out = q2k.linear(s["x"], s["w"], case["n"], bias=s["bias"], act=act, residual=s["residual"],
                         save=case["save"], const_weights=True)
        return dict(zip(("y", "z"), out)) if case["save"] else {"y": out}
    if op == "linear_bwd":
        dx, dz, dbias = q2k.linear_backward(s["dy"], s["w"], case["k"], z=s["z"], act=act,
                                            bias=case["bias"])
        return {"dx": dx, "dz": dz, "dbias": dbias} if case["bias"] else {"dx": dx, "dz": dz}
    if op == "sort":
        routes, _bad = q2k.moe_route(s["ids"], case["experts"], check=False)
        out = {"xs": q2k.moe_sort(s["x"], routes), "rows": routes.rows, "order": routes.order,
               "offsets": routes.offsets}
        if case["back"]:
            out["dx"] = q2k.moe_sort_backward(s["dxs"], routes)
        return out
    routes = q2k.Routes(s["rows"], s["order"], s["offsets"])
    if op == "combine":
        return {"y": q2k.moe_combine(s["ys"], routes, weights=s["weights"], residual=s["residual"])}
    if op == "combine_bwd":
        dys, dweights = q2k.moe_combine_backward(s["dy"], s["ys"], routes, s["weights"])
        return {"dys": dys, "dweights": dweights}
    n, k, kind = case["n"], case["k"], case["kind"]
    if kind == "linear":
        return {"y": q2k.linear(s["x"], s["w"], n, bias=s["bias"], act=act, routes=routes,
                                const_weights=True)}
    if kind == "gated":
        return {"h": q2k.gated_ffn(s["x"], s["w"], s["w2"], n, act=act, routes=routes,
                                   const_weights=True)}
    if kind == "linear_bwd":
        dx, dz, dbias = q2k.linear_backward(s["dy"], s["w"], k, z=s["z"], act=act, bias=True,
                                            routes=routes)
        return {"dx": dx, "dz": dz, "dbias": dbias}
    dx, dg, du = q2k.gated_ffn_backward(s["dy"], s["gate"], s["up"], s["w"], s["w2"], k, act=act,
                                        routes=routes)
    return {"dx": dx, "dgate": dg, "dup": du}


def work(case):
    op, m, e = case["op"], case["m"], 4 if case["dtype"] == "f32" else 2
    if op in ("linear", "linear_bwd"):
        n, k = case["n"], case["k"]
        mat = n * (k // QK) * BLOCK
        if op == "linear":
            outs = 1 + case["save"] + case["residual"]
            return {"bytes": mat + e * m * (k + n * outs) + 4 * n * case["bias"], "flops": 2 * m * n * k}
        outs = 2 + (case["act"] != "none")
        return {"bytes": mat + e * m * (k + n * outs) + 4 * n * case["bias"], "flops": 2 * m * n * k}
    r = m * case["top_k"]
    if op == "sort":
        way = e * (m + r) * case["k"]
        return {"bytes": (1 + case["back"]) * way + 12 * r + 4 * (case["experts"] + 1),
                "flops": r * case["k"] if case["back"] else r}
    if op == "combine":
        n = case["n"]
        return {"bytes": e * (r + m * (1 + case["residual"])) * n + 4 * r * (1 + case["weights"]),
                "flops": 2 * r * n}
    if op == "combine_bwd":
        n = case["n"]
        return {"bytes": e * (2 * r + m) * n + 12 * r, "flops": 3 * r * n}
    n, k, kind = case["n"], case["k"], case["kind"]
    each = 2 if kind.startswith("gated") else 1
    mats = min(r, case["experts"]) * each * n * (k // QK) * BLOCK
    acts = {"linear": k + n, "gated": k + n, "linear_bwd": k + (2 + (case["act"] != "none")) * n,
            "gated_bwd": k + 5 * n}[kind]
    return {"bytes": mats + e * r * acts, "flops": 2 * each * r * n * k}


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_rows(w, n, k):
    """float64 [n, k]: weight 128 h + 32 j + 16 s + l of a block from its bytes."""
    raw = w.view(n, k // QK, BLOCK)
    half = raw[..., 80:].contiguous().view(torch.float16).double()
    out = torch.empty((n, k // QK, QK), dtype=torch.float64, device=w.device)
    for h in range(2):
        for j in range(4):
            for s in range(2):
                byte = raw[..., 8 * h + 2 * j + s].long().unsqueeze(-1)
                q = (raw[..., 16 + 32 * h + 16 * s:][..., :16].long() // 4 ** j) % 4
                at = 128 * h + 32 * j + 16 * s
                out[..., at:at + 16] = half[..., :1] * (byte % 16) * q - half[..., 1:] * (byte // 16)
    return out.view(n, k)


def _exact_act(g, act):
    """(value, slope) in 64 bits."""
    if act == "none":
        return g, torch.ones_like(g)
    if act == "silu":
        sg = torch.sigmoid(g)
        return g * sg, sg + g * sg * torch.sigmoid(-g)
    z = GELU_C * (g + GELU_A * g ** 3)
    p = torch.sigmoid(2 * z)                       # (1 + tanh z) / 2
    return g * p, p + g * 2 * p * torch.sigmoid(-2 * z) * GELU_C * (1 + 3 * GELU_A * g ** 2)


def _exact_routes(ids, experts):
    """(rows, order, offsets) from a list of the places of each expert in turn."""
    flat = ids.reshape(-1).tolist()
    places = [[] for _ in range(experts + 1)]
    for i, e in enumerate(flat):
        places[e if 0 <= e < experts else experts].append(i)
    order = [i for p in places for i in p]
    rows = [0] * len(order)
    for p, i in enumerate(order):
        rows[i] = p
    offsets = [0]
    for p in places[:-1]:
        offsets.append(offsets[-1] + len(p))
    make = lambda v: torch.tensor(v, dtype=torch.int32, device=ids.device)  # noqa: E731
    return make(rows).view(ids.shape), make(order), make(offsets)


def _exact_bwd(dy, z, act):
    return dy.double() * (1.0 if act == "none" else _exact_act(z.double(), act)[1])


def _exact_experts(s):
    case = s["case"]
    n, k, act, kind = case["n"], case["k"], case["act"], case["kind"]
    mat = n * (k // QK) * BLOCK
    parts, dbias = [], []
    d = [s["dy"].double()] if "dy" in s else []
    if kind == "linear_bwd":
        d = [_exact_bwd(s["dy"], s["z"], act)]
    if kind == "gated_bwd":
        value, slope = _exact_act(s["gate"].double(), act)
        d = [d[0] * s["up"].double() * slope, d[0] * value]
    for e in range(case["experts"]):
        lo, hi = int(s["offsets"][e]), int(s["offsets"][e + 1])
        w = [_exact_rows(s[name][e * mat:(e + 1) * mat], n, k)
             for name in ("w", "w2") if name in s and hi > lo]
        if kind == "linear_bwd":
            dbias.append(d[0][lo:hi].sum(0))
        if hi == lo:
            continue
        if kind == "linear":
            z = s["x"][lo:hi].double() @ w[0].T
            parts.append(_exact_act(z if s["bias"] is None else z + s["bias"][e].double(), act)[0])
        elif kind == "gated":
            x = s["x"][lo:hi].double()
            parts.append(_exact_act(x @ w[0].T, act)[0] * (x @ w[1].T))
        else:
            parts.append(sum(g[lo:hi] @ v for g, v in zip(d, w)))
    out = torch.cat(parts)
    if kind == "linear":
        return {"y": out}
    if kind == "gated":
        return {"h": out}
    if kind == "linear_bwd":
        return {"dx": out, "dz": d[0], "dbias": torch.stack(dbias)}
    return {"dx": out, "dgate": d[0], "dup": d[1]}


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "linear":
        z = s["x"].double() @ _exact_rows(s["w"], case["n"], case["k"]).T
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "linear_bwd":
        dz = _exact_bwd(s["dy"], s["z"], case["act"])
        out = {"dx": dz @ _exact_rows(s["w"], case["n"], case["k"]), "dz": dz}
        return dict(out, dbias=dz.sum(0)) if case["bias"] else out
    if op == "experts":
        return _exact_experts(s)
    top_k = case["top_k"]
    if op == "sort":
        rows, order, offsets = _exact_routes(s["ids"], case["experts"])
        xs = torch.zeros((m * top_k, case["k"]), dtype=torch.float64, device="cuda")
        end = int(offsets[-1])
        xs[:end] = s["x"][(order[:end] // top_k).long()].double()
        out = {"xs": xs, "rows": rows, "order": order, "offsets": offsets}
        if case["back"]:
            dx = torch.zeros((m, case["k"]), dtype=torch.float64, device="cuda")
            dx.index_add_(0, (order[:end] // top_k).long(), s["dxs"][:end].double())
            out["dx"] = dx
        return out
    end, order, n = int(s["offsets"][-1]), s["order"].long(), case["n"]
    token = order[:end] // top_k
    if op == "combine":
        y = torch.zeros((m, n), dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            y += s["residual"].double()
        part = s["ys"][:end].double()
        if s["weights"] is not None:
            part = part * s["weights"].view(-1)[order[:end]].double().unsqueeze(-1)
        return {"y": y.index_add_(0, token, part)}
    dy = s["dy"].double()[token]
    dys = torch.zeros((m * top_k, n), dtype=torch.float64, device="cuda")
    dys[:end] = s["weights"].view(-1)[order[:end]].double().unsqueeze(-1) * dy
    dweights = torch.zeros(m * top_k, dtype=torch.float64, device="cuda")
    dweights[order[:end]] = (dy * s["ys"][:end].double()).sum(-1)
    return {"dys": dys, "dweights": dweights.view(m, top_k)}
