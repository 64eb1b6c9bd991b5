"""Cases that measure the operators of training through an MoE block: the
products grouped by expert (forward, data gradient, weight gradient), the
SwiGLU between them, the norms before and after the block with gate, dropout
and residual scale, and counter-based dropout by itself.

``run`` with ``own`` false computes them in elementary torch operations in 32
bits, rounded once at the end; with ``own`` true it makes the calls of
``combine_symmetric_heap_gb300``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # gate product of a decode step: 1024 tokens to 8 of 256 experts, about 32 rows an expert
        {"name": "product decode", "op": "product", "dtype": "bf16", "trans": False, "groups": 256, "rows": 8192, "c": 7168, "f": 2048, "skew": 0.0, "holes": 0},
        # gate product of a prefill: 8192 tokens to 8 of 256 experts, 256 +- 16 rows an expert
        {"name": "product prefill", "op": "product", "dtype": "bf16", "trans": False, "groups": 256, "rows": 65536, "c": 7168, "f": 2048, "skew": 0.0, "holes": 0},
        # data gradient of the down product, few large experts: 16384 tokens to 2 of 8 (the largest work)
        {"name": "product data gradient", "op": "product", "dtype": "bf16", "trans": True, "groups": 8, "rows": 32768, "c": 4096, "f": 14336, "skew": 0.0, "holes": 0},
        # weight gradient of the gate product, many experts of about 256 rows
        {"name": "weight gradient prefill", "op": "wgrad", "dtype": "bf16", "groups": 256, "rows": 65536, "c": 7168, "f": 2048, "skew": 0.0, "holes": 0},
        # weight gradient under uneven routing, odd counts and experts without rows, 16-bit floats
        {"name": "weight gradient uneven", "op": "wgrad", "dtype": "fp16", "groups": 24, "rows": 9001, "c": 1032, "f": 520, "skew": 1.0, "holes": 3},
        # SwiGLU of a prefill's rows with the routing weights
        {"name": "swiglu prefill", "op": "swiglu", "dtype": "bf16", "rows": 65536, "cols": 2048},
        # its gradient at a wide expert
        {"name": "swiglu gradient", "op": "swiglu_bwd", "dtype": "bf16", "rows": 32768, "cols": 14336},
        # the norms around a block for one token of a decode step: only latency counts
        {"name": "norms one token", "op": "norms", "dtype": "bf16", "rows": 1, "cols": 7168, "gate": 1, "act": "none", "p": 0.0},
        # end of a block and norm of the next one in training, gate for each sequence, dropout
        {"name": "norms train", "op": "norms", "dtype": "bf16", "rows": 16384, "cols": 4096, "gate": 8, "act": "tanh", "p": 0.1},
        # the gradient of that, at the widest hidden size, one gate for all tokens
        {"name": "norms gradient", "op": "norms_bwd", "dtype": "bf16", "rows": 8192, "cols": 7168, "gate": 1, "act": "sigmoid", "p": 0.1},
        # dropout of a training batch's activations onto the residual stream
        {"name": "dropout train", "op": "dropout", "dtype": "bf16", "rows": 16384, "cols": 4096, "p": 0.1, "residual": True},
        # dropout of a ragged batch in 32 bits, odd sizes
        {"name": "dropout odd", "op": "dropout", "dtype": "fp32", "rows": 4099, "cols": 1001, "p": 0.25, "residual": False},
    ]


def _spread(rng, lo, hi, step=1):
    """A size spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return _size(max(step, int(round(v / step)) * step))


def _size(v):
    return v + 8 if v == 3072 else v


MOST_PRODUCT = 32768 * 4096 * 14336   # multiply-adds of the largest listed case
MOST_WEIGHTS = 256 * 7168 * 2048      # weight elements of the largest listed case
MOST_ELEMENTS = 32768 * 14336


def draw(rng):
    op = rng.choice(["product", "product", "wgrad", "swiglu", "swiglu_bwd", "norms", "norms_bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op in ("product", "wgrad"):
        trans = op == "product" and rng.random() < 0.5
        groups = _spread(rng, 1, 256)
        rows = _spread(rng, 1, 65536)
        c = _spread(rng, 128, 7168, 8)
        f = _spread(rng, 128, 14336, 8 if trans or op == "wgrad" else 1)
        while groups * c * f > MOST_WEIGHTS or rows * c * f > MOST_PRODUCT:
            f = max(128, _size(f // 16 * 8))
            if f == 128:
                c = max(128, _size(c // 16 * 8))
        case = {"op": op, "dtype": dtype, "groups": groups, "rows": rows, "c": c, "f": f,
                "skew": rng.choice([0.0, 0.0, 1.0]) if groups <= 64 else 0.0,
                "holes": rng.randrange(0, groups // 4 + 1) if groups <= 64 else 0}
        if op == "product":
            case["trans"] = trans
        return case
    if op in ("swiglu", "swiglu_bwd"):
        cols = _spread(rng, 128, 14336)
        rows = min(_spread(rng, 1, 65536), _size(MOST_ELEMENTS // cols))
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": rows, "cols": cols}
    cols = _spread(rng, 128, 7168, rng.choice([1, 8]))
    if op == "dropout":
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": _spread(rng, 1, 16384), "cols": cols,
                "p": rng.choice([0.05, 0.1, 0.25, 0.5]), "residual": rng.random() < 0.5}
    rows = _spread(rng, 1, 16384)
    kind = rng.choice(["all", "sequence", "token"])
    if kind == "sequence":
        gate = rng.choice([2, 4, 8])
        rows = _size(max(1, rows // gate) * gate)
    else:
        gate = 1 if kind == "all" else rows
    return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "rows": rows, "cols": cols, "gate": gate,
            "act": rng.choice(["none", "sigmoid", "tanh"]), "p": rng.choice([0.0, 0.1])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _stream(gen, rows, cols, dtype):
    """Rows of a residual stream: token norms that differ by a few times."""
    t = torch.randn((rows, cols), generator=gen, device="cuda")
    t *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device="cuda"))
    return t.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    rows = case["rows"]
    if case["op"] in ("product", "wgrad"):
        G, C, F = case["groups"], case["c"], case["f"]
        logits = case["skew"] * torch.randn(G, generator=gen, device="cuda")
        if case["holes"]:
            logits[torch.randperm(G, generator=gen, device="cuda")[:case["holes"]]] = -math.inf
        expert = torch.multinomial(torch.softmax(logits, 0), rows, replacement=True, generator=gen)
        cnt = torch.bincount(expert, minlength=G)
        s["cnt"] = cnt.to(torch.int32)
        s["off"] = (torch.cumsum(cnt, 0) - cnt).to(torch.int32)
        s["most"] = int(cnt.max())
        if case["op"] == "product":
            s["x"] = _normal(gen, (rows, C), dt)
            s["w"] = _normal(gen, (G, C, F) if case["trans"] else (G, F, C), dt, 0.02)
            s["out"] = torch.empty((rows, F), device="cuda", dtype=dt)
        else:
            s["x"] = _normal(gen, (rows, C), dt)
            s["dy"] = _normal(gen, (rows, F), dt, 0.1)
            s["dw"] = torch.empty((G, F, C), device="cuda", dtype=dt)
        return s
    cols = case["cols"]
    if case["op"] in ("swiglu", "swiglu_bwd"):
        s["g"] = _normal(gen, (rows, cols), dt, 1.5)
        s["u"] = _normal(gen, (rows, cols), dt, 1.5)
        s["row_w"] = torch.rand(rows, generator=gen, device="cuda")
        if case["op"] == "swiglu":
            s["h"] = torch.empty((rows, cols), device="cuda", dtype=dt)
        else:
            s["dh"] = _normal(gen, (rows, cols), dt, 0.5)
            s["dg"] = torch.empty((rows, cols), device="cuda", dtype=dt)
            s["du"] = torch.empty((rows, cols), device="cuda", dtype=dt)
            s["d_row_w"] = torch.empty(rows, device="cuda")
        return s
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 0xD1B54A32D192ED03) & 0x7FFFFFFFFFFFFFFF
    s["offset"] = 7 + seed
    if case["op"] == "dropout":
        s["x"] = _normal(gen, (rows, cols), dt)
        s["res"] = _normal(gen, (rows, cols), dt) if case["residual"] else None
        s["y"] = torch.empty((rows, cols), device="cuda", dtype=dt)
        return s
    s["scale"] = 0.7
    s["o"] = _stream(gen, rows, cols, dt)
    s["w_post"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    s["w_pre"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    s["gate_t"] = _normal(gen, (case["gate"], cols), dt, 0.8)
    if case["op"] == "norms":
        s["x"] = _stream(gen, rows, cols, dt)
        s["y"] = torch.empty((rows, cols), device="cuda", dtype=dt)
        s["h"] = torch.empty((rows, cols), device="cuda", dtype=dt)
        s["rstd_post"] = torch.empty(rows, device="cuda")
        s["rstd_pre"] = torch.empty(rows, device="cuda")
        return s
    s["y"] = _stream(gen, rows, cols, dt)
    s["rstd_post"] = torch.rsqrt(s["o"].float().square().mean(1) + EPS)
    s["rstd_pre"] = torch.rsqrt(s["y"].float().square().mean(1) + EPS)
    s["dy"] = _normal(gen, (rows, cols), dt)
    s["dh"] = _normal(gen, (rows, cols), dt)
    for name, like in (("dx", "y"), ("do", "o"), ("dw_pre", "w_pre"), ("dw_post", "w_post"), ("dgate", "gate_t")):
        s[name] = torch.empty_like(s[like])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return {"product": _product, "wgrad": _wgrad, "swiglu": _swiglu, "swiglu_bwd": _swiglu_bwd,
            "norms": _norms, "norms_bwd": _norms_bwd, "dropout": _dropout}[s["op"]](s)


def _own(s):
    import combine_symmetric_heap_gb300 as sm

    op = s["op"]
    if op == "product":
        sm.moe_grouped_matmul(s["x"], s["w"], s["cnt"], s["off"], s["out"], trans_w=s["trans"])
        return s["out"]
    if op == "wgrad":
        sm.moe_grouped_wgrad(s["dy"], s["x"], s["cnt"], s["off"], s["dw"])
        return s["dw"]
    if op == "swiglu":
        sm.moe_swiglu_rows(s["g"], s["u"], s["h"], row_w=s["row_w"])
        return s["h"]
    if op == "swiglu_bwd":
        sm.moe_swiglu_rows_bwd(s["g"], s["u"], s["dh"], s["dg"], s["du"], row_w=s["row_w"], d_row_w=s["d_row_w"])
        return {"dg": s["dg"], "du": s["du"], "d_row_w": s["d_row_w"]}
    if op == "dropout":
        sm.moe_dropout(s["x"], s["y"], s["p"], s["seed"], s["offset"], residual=s["res"])
        return s["y"]
    block = dict(o=s["o"], w_post=s["w_post"], gate=s["gate_t"], gate_act=s["act"], scale=s["scale"], p=s["p"],
                 seed=s["seed"], offset=s["offset"], w_pre=s["w_pre"], rstd_post=s["rstd_post"], rstd_pre=s["rstd_pre"])
    if op == "norms":
        sm.moe_block_norm(s["x"], y=s["y"], h=s["h"], eps=EPS, **block)
        return {k: s[k] for k in ("y", "h", "rstd_post", "rstd_pre")}
    work = torch.empty(sm.moe_block_norm_workspace(s["rows"], s["cols"], s["gate"]), dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=s["dy"], dh=s["dh"], y=s["y"], dx=s["dx"], do=s["do"], dw_pre=s["dw_pre"],
                          dw_post=s["dw_post"], dgate=s["dgate"], work=work, **block)
    return {k: s[k] for k in ("dx", "do", "dw_pre", "dw_post", "dgate")}


# The products in plain form: the groups' rows padded to the longest group,
# one batched product in 32 bits, the rows taken back.
def _padded(s, t):
    at = torch.arange(s["most"], device="cuda")
    row = (s["off"].long()[:, None] + at).clamp(max=s["rows"] - 1)
    return t[row].float() * (at < s["cnt"][:, None]).unsqueeze(2)


def _product(s):
    w = s["w"].float()
    y = torch.bmm(_padded(s, s["x"]), w if s["trans"] else w.transpose(1, 2))
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    group = torch.searchsorted(s["off"], row, right=True) - 1
    return y[group, row - s["off"][group]].to(s["x"].dtype)


def _wgrad(s):
    return torch.bmm(_padded(s, s["dy"]).transpose(1, 2), _padded(s, s["x"])).to(s["x"].dtype)


def _swiglu(s):
    g = s["g"].float()
    return (s["row_w"][:, None] * (g / (1 + torch.exp(-g))) * s["u"].float()).to(s["g"].dtype)


def _swiglu_bwd(s):
    g, u, dh, w = s["g"].float(), s["u"].float(), s["dh"].float(), s["row_w"][:, None]
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    dt = s["g"].dtype
    return {"dg": (w * dh * u * (sig * (1 + g * (1 - sig)))).to(dt), "du": (w * dh * silu).to(dt), "d_row_w": (dh * silu * u).sum(1)}


# Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
# numbers: as easy as 1, 2, 3", SC 2011): block i of a stream gives elements
# 4i .. 4i+3.  int64 holds the 32-bit words; products wrap modulo 2^64.
M32 = 0xFFFFFFFF


def _philox(seed, offset, n):
    i = torch.arange((n + 3) // 4, device="cuda")
    c0, c1 = i & M32, i >> 32
    c2, c3 = torch.full_like(i, offset & M32), torch.full_like(i, offset >> 32)
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _kept(s):
    """1 / (1 - p) where an element is kept, else 0."""
    keep = _philox(s["seed"], s["offset"], s["rows"] * s["cols"]) >= int(s["p"] * 2 ** 32)
    return keep.reshape(s["rows"], s["cols"]).float() * (1 / (1 - s["p"]))


def _dropout(s):
    y = s["x"].float() * _kept(s)
    return (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)


def _gated(s):
    g = s["gate_t"].float()
    a = {"none": g, "sigmoid": 1 / (1 + torch.exp(-g)), "tanh": torch.tanh(g)}[s["act"]]
    slope = {"none": torch.ones_like(a), "sigmoid": a * (1 - a), "tanh": 1 - a * a}[s["act"]]
    each = s["rows"] // s["gate"]
    return a.repeat_interleave(each, 0), slope


def _norms(s):
    x, o, dt = s["x"].float(), s["o"].float(), s["x"].dtype
    rstd_post = 1 / torch.sqrt((o * o).mean(1) + EPS)
    b = o * rstd_post[:, None] * s["w_post"].float() * _gated(s)[0]
    if s["p"]:
        b = b * _kept(s)
    y = x + s["scale"] * b
    rstd_pre = 1 / torch.sqrt((y * y).mean(1) + EPS)
    return {"y": y.to(dt), "h": (y * rstd_pre[:, None] * s["w_pre"].float()).to(dt), "rstd_post": rstd_post, "rstd_pre": rstd_pre}


def _norms_bwd(s):
    dt, cols, G = s["y"].dtype, s["cols"], s["gate"]
    y, o, dh = s["y"].float(), s["o"].float(), s["dh"].float()
    yn, on = y * s["rstd_pre"][:, None], o * s["rstd_post"][:, None]
    t = dh * s["w_pre"].float()
    dx = s["dy"].float() + s["rstd_pre"][:, None] * (t - yn * (t * yn).mean(1, keepdim=True))
    a, slope = _gated(s)
    db = s["scale"] * dx
    if s["p"]:
        db = db * _kept(s)
    n = on * s["w_post"].float()
    dn = db * a
    t = dn * s["w_post"].float()
    do = s["rstd_post"][:, None] * (t - on * (t * on).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "do": do.to(dt), "dw_pre": (dh * yn).sum(0).to(dt), "dw_post": (dn * on).sum(0).to(dt),
            "dgate": ((db * n).reshape(G, -1, cols).sum(1) * slope).to(dt)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    b, rows, op = BYTES[case["dtype"]], case["rows"], case["op"]
    if op in ("product", "wgrad"):
        G, C, F = case["groups"], case["c"], case["f"]
        flops = 2 * rows * C * F
        if op == "wgrad":  # every group's gradient is written, zeros where it has no rows
            return {"bytes": b * (rows * (C + F) + G * C * F), "flops": flops}
        # weights of the groups that have rows: under even routing the expected number of them
        live = G - case["holes"]
        used = live * (1 - (1 - 1 / live) ** rows) if live > 1 else live
        return {"bytes": b * (rows * (C + F) + used * C * F), "flops": flops}
    n = rows * case["cols"]
    if op == "swiglu":
        return {"bytes": 3 * n * b + 4 * rows, "flops": 6 * n}
    if op == "swiglu_bwd":
        return {"bytes": 5 * n * b + 8 * rows, "flops": 14 * n}
    if op == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * n * b, "flops": 2 * n}
    gate = case["gate"] * case["cols"]
    if op == "norms":
        return {"bytes": b * (4 * n + 2 * case["cols"] + gate) + 8 * rows, "flops": 12 * n}
    return {"bytes": b * (6 * n + 4 * case["cols"] + 2 * gate) + 8 * rows, "flops": 30 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _mask64(s):
    """Kept elements from the generator's definition, in unsigned 64-bit words."""
    n = s["rows"] * s["cols"]
    u = np.uint64
    low, high = u(0xFFFFFFFF), u(32)
    keep = np.empty(((n + 3) // 4, 4), dtype=bool)
    for at in range(0, len(keep), 1 << 16):
        block = np.arange(at, min(at + (1 << 16), len(keep)), dtype=u)
        ctr = [block & low, block >> high, np.full_like(block, s["offset"] & M32), np.full_like(block, s["offset"] >> 32)]
        key = [s["seed"] & M32, (s["seed"] >> 32) & M32]
        for r in range(10):
            left, right = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
            ctr = [(right >> high) ^ ctr[1] ^ u(key[0]), right & low, (left >> high) ^ ctr[3] ^ u(key[1]), left & low]
            key = [(key[0] + 0x9E3779B9) & M32, (key[1] + 0xBB67AE85) & M32]
        for k in range(4):
            keep[at:at + len(block), k] = ctr[k] >= u(int(s["p"] * 4294967296.0))
    kept = torch.from_numpy(keep.reshape(-1)[:n]).cuda()
    return kept.reshape(s["rows"], s["cols"]).double() / (1.0 - s["p"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("product", "wgrad"):
        cnt, off = s["cnt"].tolist(), s["off"].tolist()
        if op == "product":
            out = torch.zeros((case["rows"], case["f"]), device="cuda", dtype=torch.float64)
        else:
            out = torch.zeros((case["groups"], case["f"], case["c"]), device="cuda", dtype=torch.float64)
        for e, (n, at) in enumerate(zip(cnt, off)):
            if not n:
                continue
            x = s["x"][at:at + n].double()
            if op == "product":
                w = s["w"][e].double()
                out[at:at + n] = x @ w if case["trans"] else x @ w.T
            else:
                out[e] = s["dy"][at:at + n].double().T @ x
        return out
    if op in ("swiglu", "swiglu_bwd"):
        g, u, w = s["g"].double(), s["u"].double(), s["row_w"].double().unsqueeze(1)
        sig = torch.sigmoid(g)
        if op == "swiglu":
            return w * u * g * sig
        dh = s["dh"].double()
        return {"dg": w * dh * u * (sig + g * sig * torch.sigmoid(-g)), "du": w * dh * g * sig,
                "d_row_w": torch.einsum("rc,rc->r", dh, g * sig * u)}
    if op == "dropout":
        y = s["x"].double() * _mask64(s)
        return y if s["res"] is None else y + s["res"].double()
    rows, cols, G = case["rows"], case["cols"], case["gate"]
    gate = s["gate_t"].double()
    act = {"none": lambda v: v, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[case["act"]](gate)
    act = act[:, None].expand(G, rows // G, cols).reshape(rows, cols)
    factor = s["scale"] * act
    if case["p"]:
        factor = factor * _mask64(s)
    o = s["o"].double()
    if op == "norms":
        ro = (o.square().mean(1) + EPS).rsqrt()
        y = torch.addcmul(s["x"].double(), factor, o * ro[:, None] * s["w_post"].double())
        ry = (y.square().mean(1) + EPS).rsqrt()
        return {"y": y, "h": y * ry[:, None] * s["w_pre"].double(), "rstd_post": ro, "rstd_pre": ry}
    ry, ro = s["rstd_pre"].double()[:, None], s["rstd_post"].double()[:, None]
    y, dh, wp, wo = s["y"].double(), s["dh"].double(), s["w_pre"].double(), s["w_post"].double()
    inner = (dh * wp * y).sum(1, keepdim=True) / cols
    dx = s["dy"].double() + ry * dh * wp - ry ** 3 * y * inner
    dn = dx * factor
    inner = (dn * wo * o).sum(1, keepdim=True) / cols
    slope = {"none": torch.ones_like(gate), "sigmoid": torch.sigmoid(gate) * torch.sigmoid(-gate),
             "tanh": torch.cosh(gate) ** -2}[case["act"]]
    # the gate's gradient by its own factor: dx * scale * mask * norm(o)
    plain = s["scale"] * (_mask64(s) if case["p"] else 1.0)
    dact = (dx * plain * o * ro * wo).reshape(G, rows // G, cols).sum(1)
    return {"dx": dx, "do": ro * dn * wo - ro ** 3 * o * inner, "dw_pre": (dh * y * ry).sum(0),
            "dw_post": (dn * o * ro).sum(0), "dgate": dact * slope}
