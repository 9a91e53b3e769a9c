"""Measured cases of the feed-forward operators on Q2_K weights.

Three operators, each over weights stored as GGML Q2_K blocks (84 bytes per 256
weights):

``gated``     h = act(x Wg^T) * (x Wu^T), the gated feed-forward block's two
              projections, activation and product; ``save`` also returns the two
              projections, which the backward pass reads.
``gated_bwd`` its backward pass with the weights frozen: dx, and the gradients of
              the two projections.
``lora``      y = x W^T + s_a (x A_a^T) B_a^T with one low-rank adapter a per
              token (or none, id -1) beside the shared projection.

``run`` computes them in elementary torch operations in 32 bits (``own`` false),
or by the calls that a user of the package makes (``own`` true).
"""

import math

import torch

own = False

QK, BLOCK = 256, 84
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    gated = {"op": "gated", "act": "silu", "save": False}
    return [
        # one token through the tiny workload's matrices: nothing but latency
        dict(gated, name="gated tiny m4", dtype="f32", m=4, n=8, k=256),
        # decode: one token through the FFN pair of the benchmark's workloads
        dict(gated, name="gated decode m1", dtype="f32", m=1, n=14336, k=4096),
        # speculative verification: sixteen draft tokens through the same block
        dict(gated, name="gated verify m16", dtype="bf16", m=16, n=14336, k=4096),
        # a short prompt and a block of odd sizes (rows that start off 16 bytes)
        dict(gated, name="gated ragged m77", dtype="bf16", m=77, n=4999, k=2816, act="gelu"),
        # a training micro-batch's forward pass, projections kept for the backward
        dict(gated, name="gated train m512", dtype="bf16", m=512, n=14336, k=4096, save=True),
        # its backward pass
        {"name": "gated bwd m512", "op": "gated_bwd", "act": "silu", "dtype": "bf16",
         "m": 512, "n": 14336, "k": 4096},
        # a few tokens' gradients through a small block of odd sizes
        {"name": "gated bwd ragged m37", "op": "gated_bwd", "act": "gelu", "dtype": "bf16",
         "m": 37, "n": 1001, "k": 1280},
        # the largest: four sequences of 512 tokens backwards
        {"name": "gated bwd m2048", "op": "gated_bwd", "act": "silu", "dtype": "bf16",
         "m": 2048, "n": 14336, "k": 4096},
        # one request's decode step through a square projection with its adapter
        {"name": "lora decode m1", "op": "lora", "dtype": "f32", "m": 1, "n": 4096, "k": 4096,
         "rank": 16, "adapters": 8, "spread": "segments"},
        # sixteen requests' tokens, adapters in any order and some without, FFN down
        {"name": "lora requests m16", "op": "lora", "dtype": "bf16", "m": 16, "n": 4096,
         "k": 14336, "rank": 16, "adapters": 16, "spread": "mixed"},
        # odd sizes, a few dozen tokens of a handful of requests
        {"name": "lora ragged m45", "op": "lora", "dtype": "bf16", "m": 45, "n": 1003, "k": 1792,
         "rank": 8, "adapters": 5, "spread": "mixed"},
        # four requests' prompts in one batch, rank 64
        {"name": "lora prompts m512", "op": "lora", "dtype": "bf16", "m": 512, "n": 7168,
         "k": 7168, "rank": 64, "adapters": 4, "spread": "segments"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "lora", "lora"])
    while True:
        m, n, k = _log_int(rng, 1, 2048), _log_int(rng, 8, 14336), QK * _log_int(rng, 1, 56)
        if m * n * k <= 512 * 14336 * 4096:
            break
    # 32-bit activations are the decode form; larger batches are held in bf16
    dtype = rng.choice(["f32", "bf16"]) if m <= 8 and op != "gated_bwd" else "bf16"
    case = {"op": op, "dtype": dtype, "m": m, "n": n, "k": k}
    if op == "lora":
        case.update(rank=8 * _log_int(rng, 1, 16), adapters=_log_int(rng, 1, 32),
                    spread=rng.choice(["segments", "mixed"]))
    else:
        case["act"] = rng.choice(["silu", "gelu"])
        if op == "gated":
            case["save"] = rng.random() < 0.5
    return case


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "lora":
        r, a = case["rank"], case["adapters"]
        s["x"], s["w"] = _tensor(gen, dt, m, k), _blocks(gen, n, k)
        s["a"] = _tensor(gen, torch.bfloat16, a, r, k, scale=1 / math.sqrt(k))
        s["b"] = _tensor(gen, torch.bfloat16, a, n, r, scale=1 / math.sqrt(r))
        s["scales"] = 0.25 + torch.rand(a, device="cuda", generator=gen)
        if case["spread"] == "segments":
            s["ids"] = (torch.arange(m, device="cuda") * a // m).to(torch.int32)
        else:
            s["ids"] = torch.randint(-1, a, (m,), device="cuda", generator=gen, dtype=torch.int32)
    else:
        s["wg"], s["wu"] = _blocks(gen, n, k), _blocks(gen, n, k)
        if case["op"] == "gated":
            s["x"] = _tensor(gen, dt, m, k)
        else:
            s["dh"] = _tensor(gen, dt, m, n, scale=0.1)
            s["gate"], s["up"] = _tensor(gen, dt, m, n, scale=1.5), _tensor(gen, dt, m, n, scale=1.5)
    return s


# ---- plain forms ---------------------------------------------------------------

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
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(GELU_C * (g + GELU_A * g * g * g)))


def _act_slope(g, act):
    if act == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return sg * (1 + g * (1 - sg))
    t = torch.tanh(GELU_C * (g + GELU_A * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * GELU_A * g * g)


def _plain(s):
    case = s["case"]
    n, k, dt = case["n"], case["k"], DTYPES[case["dtype"]]
    if case["op"] == "gated":
        x = s["x"].float()
        g, u = x @ _weights(s["wg"], n, k).T, x @ _weights(s["wu"], n, k).T
        out = {"h": (_act(g, case["act"]) * u).to(dt)}
        if case["save"]:
            out["gate"], out["up"] = g.to(dt), u.to(dt)
        return out
    if case["op"] == "gated_bwd":
        dh, g, u = s["dh"].float(), s["gate"].float(), s["up"].float()
        dg, du = dh * u * _act_slope(g, case["act"]), dh * _act(g, case["act"])
        dx = dg @ _weights(s["wg"], n, k) + du @ _weights(s["wu"], n, k)
        return {"dx": dx.to(dt), "dgate": dg.to(dt), "dup": du.to(dt)}
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    m, (na, r) = x.shape[0], a.shape[:2]
    own_adapter = (s["ids"].view(m, 1) == torch.arange(na, device="cuda")).float() * s["scales"]
    t = (x @ a.view(na * r, k).T).view(m, na, r) * own_adapter.view(m, na, 1)
    y = x @ _weights(s["w"], n, k).T + t.view(m, na * r) @ b.transpose(0, 1).reshape(n, na * r).T
    return {"y": y.to(dt)}


def run(s):
    if not own:
        return _plain(s)
    import ggml_q2_quantized_gb300 as q2k
    case = s["case"]
    if case["op"] == "gated":
        out = q2k.gated_ffn(s["x"], s["wg"], s["wu"], case["n"], act=case["act"],
                            save=case["save"], const_weights=True)
        return dict(zip(("h", "gate", "up"), out)) if case["save"] else {"h": out}
    if case["op"] == "gated_bwd":
        dx, dg, du = q2k.gated_ffn_backward(s["dh"], s["gate"], s["up"], s["wg"], s["wu"],
                                            case["k"], act=case["act"])
        return {"dx": dx, "dgate": dg, "dup": du}
    y, _bad = q2k.matmul_lora(s["x"], s["w"], case["n"], s["a"], s["b"], s["ids"],
                              scales=s["scales"], const_weights=True, check=False)
    return {"y": y}


def work(case):
    m, n, k, e = case["m"], case["n"], case["k"], 4 if case["dtype"] == "f32" else 2
    mat = n * (k // QK) * BLOCK
    if case["op"] == "gated":
        return {"bytes": 2 * mat + e * m * (k + n * (3 if case["save"] else 1)),
                "flops": 4 * m * n * k}
    if case["op"] == "gated_bwd":
        return {"bytes": 2 * mat + e * m * (k + 5 * n), "flops": 4 * m * n * k}
    used = min(m, case["adapters"])
    return {"bytes": mat + e * m * (k + n) + 4 * m + 2 * used * case["rank"] * (k + n),
            "flops": 2 * m * n * k + 2 * m * case["rank"] * (k + n)}


# ---- the definitions in 64 bits --------------------------------------------------

def _exact_rows(w, n, k):
    """float64 [n, k]: weight 128 h + 32 j + 16 s + l of a block from its bytes."""
    raw = w.view(n, k // QK, BLOCK).to(torch.int64)
    half = raw[..., 80:].to(torch.uint8).contiguous().view(torch.float16).double()
    out = torch.empty((n, k // QK, QK), dtype=torch.float64, device=w.device)
    for h in range(2):
        for j in range(4):
            for s in range(2):
                byte = raw[..., 8 * h + 2 * j + s].unsqueeze(-1)
                q = (raw[..., 16 + 32 * h + 16 * s:][..., :16] // 4 ** j) % 4
                at = 128 * h + 32 * j + 16 * s
                out[..., at:at + 16] = half[..., :1] * (byte % 16) * q - half[..., 1:] * (byte // 16)
    return out.view(n, k)


def _exact_act(g, act):
    """(value, slope) in 64 bits."""
    if act == "silu":
        sg = torch.sigmoid(g)
        return g * sg, sg + g * sg * torch.sigmoid(-g)
    z = GELU_C * (g + GELU_A * g ** 3)
    p = torch.sigmoid(2 * z)                       # (1 + tanh z) / 2
    return g * p, p + g * 2 * p * torch.sigmoid(-2 * z) * GELU_C * (1 + 3 * GELU_A * g ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    n, k = case["n"], case["k"]
    if case["op"] == "gated":
        x = s["x"].double()
        g, u = x @ _exact_rows(s["wg"], n, k).T, x @ _exact_rows(s["wu"], n, k).T
        out = {"h": _exact_act(g, case["act"])[0] * u}
        return dict(out, gate=g, up=u) if case["save"] else out
    if case["op"] == "gated_bwd":
        dh, g, u = s["dh"].double(), s["gate"].double(), s["up"].double()
        value, slope = _exact_act(g, case["act"])
        dg, du = dh * u * slope, dh * value
        dx = dg @ _exact_rows(s["wg"], n, k)
        dx += du @ _exact_rows(s["wu"], n, k)
        return {"dx": dx, "dgate": dg, "dup": du}
    x = s["x"].double()
    y = x @ _exact_rows(s["w"], n, k).T
    for a in range(case["adapters"]):
        rows = (s["ids"] == a).nonzero().view(-1)
        t = x[rows] @ s["a"][a].double().T
        y[rows] += s["scales"][a].double() * (t @ s["b"][a].double().T)
    return {"y": y}
