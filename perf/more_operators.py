"""Cases that measure three operators around an MoE block: the whole layer for a
few tokens (routing, experts, combine), layer norm forward and backward with the
residual sum in the same pass, and the orthogonalising of a batch of updates by
Newton-Schulz products.

``run`` with ``own`` false computes them in elementary torch operations in 32
bits, rounded once at the end; with ``own`` true it makes the calls of
``combine_symmetric_heap_gb300``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5        # of the layer norm
NORM_EPS = 1e-7   # added to an update's norm
STEPS, COEFFS = 5, (3.4445, -4.7750, 2.0315)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token being served through two of eight wide experts: a read of their weights
        {"name": "layer one token", "op": "layer", "dtype": "bf16", "tokens": 1, "h": 4096, "i": 14336, "experts": 8, "topk": 2, "router": False, "fused": False},
        # 32 users' next tokens through eight of 256 experts each, from the router's weights on (the largest)
        {"name": "layer 32 tokens", "op": "layer", "dtype": "bf16", "tokens": 32, "h": 7168, "i": 2048, "experts": 256, "topk": 8, "router": True, "fused": False},
        # a small model's four tokens: only latency counts
        {"name": "layer small", "op": "layer", "dtype": "bf16", "tokens": 4, "h": 128, "i": 256, "experts": 4, "topk": 2, "router": True, "fused": False},
        # sizes off every power of two in 16-bit floats, gate and up rows of an expert in one matrix
        {"name": "layer odd", "op": "layer", "dtype": "fp16", "tokens": 7, "h": 1032, "i": 520, "experts": 24, "topk": 3, "router": False, "fused": True},
        # the norm in front of a block for one token of a decode step: only latency counts
        {"name": "layer norm one token", "op": "norm", "dtype": "bf16", "rows": 1, "cols": 7168, "add": True},
        # end of a block and norm of the next one over a training batch
        {"name": "layer norm train", "op": "norm", "dtype": "bf16", "rows": 16384, "cols": 4096, "add": True},
        # its gradient at a wide hidden size, the stream's own gradient added in
        {"name": "layer norm gradient", "op": "norm_bwd", "dtype": "bf16", "rows": 8192, "cols": 7168, "add": True},
        # the gradient over a ragged batch in 32 bits, odd sizes
        {"name": "layer norm gradient odd", "op": "norm_bwd", "dtype": "fp32", "rows": 4099, "cols": 1001, "add": False},
        # the update of a router's weights: one small matrix, 15 dependent products
        {"name": "orthogonalize router", "op": "orth", "dtype": "bf16", "count": 1, "f": 256, "c": 7168},
        # the updates of eight experts' gate matrices
        {"name": "orthogonalize experts", "op": "orth", "dtype": "bf16", "count": 8, "f": 2048, "c": 7168},
        # of a wide expert's down matrix, held in 32 bits as momentum is
        {"name": "orthogonalize momentum", "op": "orth", "dtype": "bf16", "count": 1, "f": 4096, "c": 14336, "momentum": True},
        # tall ones off every power of two in 16-bit floats
        {"name": "orthogonalize odd", "op": "orth", "dtype": "fp16", "count": 5, "f": 1031, "c": 519},
    ]


def _spread(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


MOST_WEIGHTS = 256 * 7168 * 2048     # elements of one of the largest listed case's weights
MOST_LIVE = 160 * 7168 * 2048        # about as many as its 32 tokens read
MOST_ELEMENTS = 16384 * 4096
MOST_PRODUCTS = 8 * (4 * 2048 * 2048 * 7168 + 2 * 2048 ** 3)


def draw(rng):
    op = rng.choice(["layer", "layer", "norm", "norm_bwd", "orth"])
    if op == "layer":
        h, i = _spread(rng, 128, 7168, 8), _spread(rng, 128, 14336, 8)
        experts = _spread(rng, 2, 256)
        topk = rng.randint(1, min(8, experts))
        tokens = _spread(rng, 1, 32)
        while experts * h * i > MOST_WEIGHTS or min(experts, tokens * topk) * h * i > MOST_LIVE:
            i = max(128, i // 16 * 8)
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "tokens": tokens, "h": h, "i": i, "experts": experts,
                "topk": topk, "router": rng.random() < 0.5, "fused": rng.random() < 0.5}
    if op in ("norm", "norm_bwd"):
        cols = _spread(rng, 128, 16384, rng.choice([1, 8]))
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": min(_spread(rng, 1, 65536), max(1, MOST_ELEMENTS // cols)),
                "cols": cols, "add": rng.random() < 0.5}
    f, c, count = _spread(rng, 64, 7168), _spread(rng, 64, 7168), _spread(rng, 1, 24)
    m, n = min(f, c), max(f, c)
    count = max(1, min(count, MOST_PRODUCTS // (4 * m * m * n + 2 * m ** 3)))
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "count": count, "f": f, "c": c, "momentum": rng.random() < 0.3}
    while count * (4 * m * m * n + 2 * m ** 3) > MOST_PRODUCTS:  # both sides near the top of the range
        m, n = m // 2, n // 2
        case["f"], case["c"] = case["f"] // 2, case["c"] // 2
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _stream(gen, rows, cols, dtype):
    """Rows of a residual stream: token norms that differ by a few times, means off zero, a few large columns."""
    t = torch.randn((rows, cols), generator=gen, device="cuda")
    t *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda"))
    t += 0.3 * torch.randn((rows, 1), generator=gen, device="cuda")
    big = torch.randint(cols, (3,), generator=gen, device="cuda")
    t[:, big] *= 8
    return t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "layer":
        T, H, I, E, k = (case[n] for n in ("tokens", "h", "i", "experts", "topk"))
        s["x"] = _normal(gen, (T, H), dt)
        if case["fused"]:  # each expert's gate rows above its up rows
            both = _normal(gen, (E, 2 * I, H), dt, H ** -0.5)
            s["w_gate"], s["w_up"] = both[:, :I], both[:, I:]
        else:
            s["w_gate"], s["w_up"] = _normal(gen, (E, I, H), dt, H ** -0.5), _normal(gen, (E, I, H), dt, H ** -0.5)
        s["w_down"] = _normal(gen, (E, H, I), dt, I ** -0.5)
        if case["router"]:
            s["w_router"] = _normal(gen, (E, H), dt, H ** -0.5)
            s["logits"] = torch.empty((T, E), device="cuda")
        else:
            s["logits"] = torch.randn((T, E), generator=gen, device="cuda")
        s["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, k), device="cuda")
        s["out"] = torch.empty((T, H), device="cuda", dtype=dt)
        return s
    if case["op"] == "orth":
        # a gradient: a few strong directions over a broad rest
        count, F, C = case["count"], case["f"], case["c"]
        r = max(1, min(F, C) // 8)
        left, right = _normal(gen, (count, F, r), torch.float32), _normal(gen, (count, r, C), torch.float32)
        left *= torch.arange(1, r + 1, device="cuda") ** -0.5
        g = torch.bmm(left, right).add_(_normal(gen, (count, F, C), torch.float32, 0.5)).mul_(1e-3)
        s["g"] = g if case.get("momentum") else g.to(dt)
        s["out"] = torch.empty((count, F, C), device="cuda", dtype=dt)
        return s
    rows, cols = case["rows"], case["cols"]
    s["x"] = _stream(gen, rows, cols, dt)
    s["w_ln"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    s["b_ln"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if case["op"] == "norm":
        s["o"] = _normal(gen, (rows, cols), dt, 0.5) if case["add"] else None
        s["sum"] = torch.empty((rows, cols), device="cuda", dtype=dt) if case["add"] else None
        s["out"] = torch.empty((rows, cols), device="cuda", dtype=dt)
        return s
    x = s["x"].float()
    torch.mean(x, 1, out=s["mean"])
    torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + EPS, out=s["rstd"])
    s["dh"] = _normal(gen, (rows, cols), dt)
    s["dsum"] = _normal(gen, (rows, cols), dt) if case["add"] else None
    s["dx"] = torch.empty((rows, cols), device="cuda", dtype=dt)
    s["dw"], s["db"] = torch.empty(cols, device="cuda", dtype=dt), torch.empty(cols, device="cuda", dtype=dt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"layer": _layer, "norm": _norm, "norm_bwd": _norm_bwd, "orth": _orth}[s["op"]](s)


def _own(s):
    import combine_symmetric_heap_gb300 as sm

    def work(n):
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    op = s["op"]
    if op == "layer":
        sm.moe_few_tokens(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["logits"], s["idx"], s["w"], s["out"],
                          work(sm.moe_few_tokens_workspace(s["tokens"], s["i"], s["topk"])), w_router=s.get("w_router"))
        got = {k: s[k] for k in ("out", "idx", "w")}
        return dict(got, logits=s["logits"]) if s["router"] else got
    if op == "orth":
        sm.moe_orthogonalize(s["g"], s["out"], work(sm.moe_orthogonalize_workspace(s["count"], s["f"], s["c"])),
                             steps=STEPS, coeffs=COEFFS, eps=NORM_EPS)
        return s["out"]
    if op == "norm":
        sm.moe_layer_norm(s["x"], s["out"], w=s["w_ln"], b=s["b_ln"], add=s["o"], sum=s["sum"], mean=s["mean"],
                          rstd=s["rstd"], eps=EPS)
        got = {k: s[k] for k in ("out", "mean", "rstd")}
        return dict(got, sum=s["sum"]) if s["add"] else got
    sm.moe_layer_norm_bwd(s["dh"], s["x"], s["mean"], s["rstd"], dx=s["dx"], w=s["w_ln"], dsum=s["dsum"], dw=s["dw"],
                          db=s["db"], work=work(sm.moe_layer_norm_workspace(s["rows"], s["cols"])))
    return {k: s[k] for k in ("dx", "dw", "db")}


def _layer(s):
    x, dt = s["x"].float(), s["x"].dtype
    # a logit next to another decides which expert a token gets: added in 64 bits
    logits = (x.double() @ s["w_router"].double().T).float() if s["router"] else s["logits"]
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :s["topk"]], idx[:, :s["topk"]]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for j in range(s["topk"]):
        e = idx[:, j]
        g = torch.bmm(s["w_gate"][e].float(), x.unsqueeze(2))
        u = torch.bmm(s["w_up"][e].float(), x.unsqueeze(2))
        h = g / (1 + torch.exp(-g)) * u
        out += w[:, j:j + 1] * torch.bmm(s["w_down"][e].float(), h).squeeze(2)
    got = {"out": out.to(dt), "idx": idx.to(torch.int32), "w": w}
    return dict(got, logits=logits) if s["router"] else got


def _norm(s):
    x, dt = s["x"].float(), s["x"].dtype
    if s["add"]:
        x = x + s["o"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    got = {"out": (c * rstd[:, None] * s["w_ln"].float() + s["b_ln"].float()).to(dt), "mean": mean, "rstd": rstd}
    return dict(got, sum=x.to(dt)) if s["add"] else got


def _norm_bwd(s):
    dt = s["x"].dtype
    dh = s["dh"].float()
    n = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dh * s["w_ln"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    if s["add"]:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(dt), "dw": (dh * n).sum(0).to(dt), "db": dh.sum(0).to(dt)}


def _orth(s):
    a, b, c = COEFFS
    x = s["g"].float()
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NORM_EPS)
    tall = s["f"] > s["c"]
    for _ in range(STEPS):
        gram = torch.bmm(x.transpose(1, 2), x) if tall else torch.bmm(x, x.transpose(1, 2))
        poly = b * gram + c * torch.bmm(gram, gram)
        x = a * x + (torch.bmm(x, poly) if tall else torch.bmm(poly, x))
    return x.to(s["out"].dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "layer":
        T, H, I, E, k = (case[n] for n in ("tokens", "h", "i", "experts", "topk"))
        live = E * (1 - (1 - k / E) ** T)  # expected number of experts that some token chose
        n = b * (3 * live * H * I + 2 * T * H) + 4 * T * (E + 2 * k) + (b * E * H if case["router"] else 0)
        return {"bytes": n, "flops": 6 * T * k * H * I + (2 * T * E * H if case["router"] else 0)}
    if case["op"] == "orth":
        F, C, count = case["f"], case["c"], case["count"]
        m, n = min(F, C), max(F, C)
        # a Gram matrix and its square are symmetric: half of each
        return {"bytes": count * F * C * (b + (4 if case.get("momentum") else b)), "flops": count * STEPS * (3 * m * m * n + m ** 3)}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "norm":
        return {"bytes": b * ((4 if case["add"] else 2) * n + 2 * cols) + 8 * rows, "flops": 8 * n}
    return {"bytes": b * ((4 if case["add"] else 3) * n + 3 * cols) + 8 * rows, "flops": 14 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_layer(s, case):
    x = s["x"].double()
    logits = torch.einsum("th,eh->te", x, s["w_router"].double()) if case["router"] else s["logits"].double()
    T, k = case["tokens"], case["topk"]
    out = torch.zeros_like(x)
    chosen = []  # per token: (expert, weight), by repeated largest with the lowest index first
    for row in logits.tolist():
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        z = [math.exp(row[e] - row[order[0]]) for e in order]
        chosen.append([(e, v / math.fsum(z)) for e, v in zip(order, z)])
    for e in sorted({e for c in chosen for e, _ in c}):
        t, w = zip(*[(t, v) for t in range(T) for f, v in chosen[t] if f == e])
        rows = x[list(t)]
        g = rows @ s["w_gate"][e].double().T
        h = g * torch.sigmoid(g) * (rows @ s["w_up"][e].double().T)
        out[list(t)] += torch.tensor(w, device="cuda", dtype=torch.float64)[:, None] * (h @ s["w_down"][e].double().T)
    got = {"out": out, "idx": torch.tensor([[e for e, _ in c] for c in chosen], device="cuda", dtype=torch.int32),
           "w": torch.tensor([[v for _, v in c] for c in chosen], device="cuda", dtype=torch.float64)}
    return dict(got, logits=logits) if case["router"] else got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        return _exact_layer(s, case)
    if case["op"] == "orth":
        F, C = case["f"], case["c"]
        if case["count"] * min(F, C) ** 2 * max(F, C) * 6 * STEPS > 12e12:  # 64-bit products run at about 1 TFLOP/s
            return None
        a, b, c = COEFFS
        out = torch.empty((case["count"], F, C), device="cuda", dtype=torch.float64)
        for i in range(case["count"]):
            x = s["g"][i].double()
            x = x if F <= C else x.T
            x = x / (torch.linalg.vector_norm(x) + NORM_EPS)
            for _ in range(STEPS):  # without the square of the Gram matrix
                y = (x @ x.T) @ x
                x = a * x + b * y + c * ((x @ x.T) @ y)
            out[i] = x if F <= C else x.T
        return out
    x = s["x"].double()
    if case["op"] == "norm":
        if case["add"]:
            x = x + s["o"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        y = torch.addcmul(s["b_ln"].double(), (x - mean[:, None]) * rstd[:, None], s["w_ln"].double())
        got = {"out": y, "mean": mean, "rstd": rstd}
        return dict(got, sum=x) if case["add"] else got
    dh, w, rstd = s["dh"].double(), s["w_ln"].double(), s["rstd"].double()[:, None]
    d = x - s["mean"].double()[:, None]
    inner = torch.einsum("rc,rc,c->r", dh, d, w)[:, None] / case["cols"]
    dx = rstd * dh * w - rstd * (dh @ w)[:, None] / case["cols"] - rstd ** 3 * d * inner
    if case["add"]:
        dx += s["dsum"].double()
    return {"dx": dx, "dw": torch.einsum("rc,rc->c", dh, d * rstd), "db": dh.sum(0)}
