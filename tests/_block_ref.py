"""Definitions in 64 bits of the operators of training through an MoE block,
and the error bounds that follow from their number formats.

Every definition also returns the sum of the absolute values of each result's
terms.  An fp32 evaluation is off by at most a small multiple of 2^-24 of that
sum: EVAL covers about 170 roundings (the elementary functions' few ulps, a
few dozen products, a tree sum over a row); a result in 16 bits is off by half
a unit in the last place of its own on top (UNIT)."""
from __future__ import annotations

import numpy as np
import torch

EVAL = 1e-5
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
TINY = {torch.bfloat16: 1e-37, torch.float16: 2.0 ** -24, torch.float32: 1e-37}  # spacing of the smallest values


def assert_within(got, ref, mag, what, eval_=EVAL):
    dt = got.dtype
    got, ref, mag = got.double(), ref.double(), mag.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bound = UNIT[dt] * ref.abs() + eval_ * mag * (1 + UNIT[dt]) + TINY[dt]
    bad = ~((got - ref).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), got[bad][:4].tolist(), ref[bad][:4].tolist(), bound[bad][:4].tolist())


# ---------------------------------------------------------------- products
def product_bound(k: int) -> float:
    """Error of k products added by the tensor cores into an fp32 accumulator,
    relative to the sum of their absolute values: each step of 16 truncates
    twice at most (inside, and into the accumulator)."""
    return (k / 8 + 8) * 2.0 ** -23


def groups_of(counts, slots=1, gap=0, device="cuda"):
    """cnt, off int32 [slots, G / slots] and rows a slot needs, with `gap`
    unused rows before, between and after the groups."""
    each = len(counts) // slots
    cnt = torch.tensor(counts, dtype=torch.int32).view(slots, each)
    off = gap + torch.cumsum(cnt + gap, 1, dtype=torch.int32) - cnt - gap
    rows = int((off + cnt).max()) + gap
    return cnt.to(device), off.to(device), rows


def each_group(cnt, off):
    slots, each = cnt.shape
    c, o = cnt.tolist(), off.tolist()
    for e in range(slots * each):
        d, j = divmod(e, each)
        yield e, d, o[d][j], c[d][j]


def ref_product(x, w, cnt, off, trans):
    x = x.double()
    out = torch.zeros(*x.shape[:2], w.shape[2] if trans else w.shape[1], dtype=torch.float64, device=x.device)
    mag, live = torch.zeros_like(out), torch.zeros(x.shape[:2], dtype=torch.bool, device=x.device)
    for e, d, at, n in each_group(cnt, off):
        if n:
            m = w[e].double() if trans else w[e].double().T
            rows = x[d, at:at + n]
            out[d, at:at + n] = rows @ m
            mag[d, at:at + n] = rows.abs() @ m.abs()
            live[d, at:at + n] = True
    return out, mag, live


def ref_wgrad(dy, x, cnt, off):
    G = cnt.numel()
    out = torch.zeros(G, dy.shape[2], x.shape[2], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, d, at, n in each_group(cnt, off):
        if n:
            a, b = dy[d, at:at + n].double(), x[d, at:at + n].double()
            out[e] = a.T @ b
            mag[e] = a.abs().T @ b.abs()
    return out, mag


# ---------------------------------------------------------------- swiglu
def ref_swiglu(g, u, w):
    g, u, w = g.double(), u.double(), w.double().unsqueeze(-1)
    return w * g * torch.sigmoid(g) * u


def ref_swiglu_bwd(g, u, dh, w):
    g, u, dh, w = g.double(), u.double(), dh.double(), w.double().unsqueeze(-1)
    s = torch.sigmoid(g)
    dg = w * dh * u * s * (1 + g * (1 - s))
    dg_mag = (w * dh * u * s).abs() * (1 + g.abs() * (1 - s))
    du, terms = w * dh * g * s, dh * g * s * u
    return (dg, dg_mag), (du, du.abs()), (terms.sum(-1), terms.abs().sum(-1))


# ---------------------------------------------------------------- dropout
def words(seed: int, offset: int, n: int) -> np.ndarray:
    """Words 0..n-1 of the stream, one Python integer operation at a time for
    the constants, numpy for the counters (Philox 4x32, 10 rounds)."""
    m = 0xFFFFFFFF
    i = np.arange((n + 3) // 4, dtype=np.uint64)
    c = [i & np.uint64(m), i >> np.uint64(32), np.full_like(i, offset & m), np.full_like(i, offset >> 32)]
    k = [seed & m, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & np.uint64(m),
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & np.uint64(m)]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return np.stack(c, 1).reshape(-1)[:n]


def kept(seed, offset, shape, p, device="cuda"):
    n = int(np.prod(shape))
    return torch.from_numpy(words(seed, offset, n) >= np.uint64(int(p * 2 ** 32))).to(device).view(shape)


# ---------------------------------------------------------------- norms
def _act(name, g):
    a = {"none": g, "sigmoid": torch.sigmoid(g), "tanh": torch.tanh(g)}[name]
    s = {"none": torch.ones_like(g), "sigmoid": torch.sigmoid(g) * torch.sigmoid(-g), "tanh": 1 - torch.tanh(g) ** 2}[name]
    return a, s


def ref_norm(x, o=None, w_post=None, gate=None, gate_act="none", scale=1.0, p=0.0, seed=0, offset=0, w_pre=None,
             post_norm=True, eps=1e-6):
    """y, h, rstd_post, rstd_pre and the terms' sizes of y and h."""
    x = x.double()
    R, C = x.shape
    y, mag, ro = x, x.abs(), None
    if o is not None:
        o = o.double()
        ro = (o.square().mean(1) + eps).rsqrt() if post_norm else torch.ones(R, dtype=x.dtype, device=x.device)
        b = o * ro[:, None]
        if w_post is not None:
            b = b * w_post.double()
        if gate is not None:
            b = b * _act(gate_act, gate.double())[0].repeat_interleave(R // gate.shape[0], 0)
        if p:
            b = torch.where(kept(seed, offset, (R, C), p, x.device), b / (1 - p), torch.zeros_like(b))
        y = x + scale * b
        mag = x.abs() + (scale * b).abs()
    ry = (y.square().mean(1) + eps).rsqrt()
    wp = torch.ones(C, dtype=x.dtype, device=x.device) if w_pre is None else w_pre.double()
    return dict(y=y, h=y * ry[:, None] * wp, rstd_post=ro, rstd_pre=ry), dict(y=mag, h=mag * ry[:, None] * wp.abs())


def ref_norm_bwd(dy, dh, y, o, w_post, gate, gate_act, scale, p, seed, offset, w_pre, rstd_post, rstd_pre, post_norm=True):
    """{name: (gradient, size of its terms)}"""
    lead = dy if dy is not None else dh
    R, C = lead.shape
    one = lambda w: torch.ones(C, dtype=torch.float64, device=lead.device) if w is None else w.double()  # noqa: E731
    out = {}
    dx = torch.zeros(R, C, dtype=torch.float64, device=lead.device) if dy is None else dy.double()
    mag = dx.abs()
    if dh is not None:
        t, yn = dh.double() * one(w_pre), y.double() * rstd_pre.double()[:, None]
        dx = dx + rstd_pre.double()[:, None] * (t - yn * (t * yn).mean(1, keepdim=True))
        mag = mag + rstd_pre.double()[:, None] * (t.abs() + yn.abs() * (t * yn).abs().mean(1, keepdim=True))
        d = dh.double() * yn
        out["dw_pre"] = (d.sum(0), d.abs().sum(0))
    out["dx"] = (dx, mag)
    if o is not None:
        ro = rstd_post.double()[:, None] if post_norm else torch.ones(R, 1, dtype=torch.float64, device=lead.device)
        on, w = o.double() * ro, one(w_post)
        m = torch.full((R, C), scale, dtype=torch.float64, device=lead.device)
        if p:
            m = m * kept(seed, offset, (R, C), p, lead.device) / (1 - p)
        G = 1 if gate is None else gate.shape[0]
        a, s = (torch.ones(1, C, dtype=torch.float64, device=lead.device),) * 2 if gate is None else _act(gate_act, gate.double())
        f = m * a.repeat_interleave(R // G, 0)
        dn, dn_mag = dx * f, mag * f.abs()
        t, t_mag = dn * w, dn_mag * w.abs()
        if post_norm:
            out["do"] = (ro * (t - on * (t * on).mean(1, keepdim=True)),
                         ro * (t_mag + on.abs() * (t_mag * on.abs()).mean(1, keepdim=True)))
            out["dw_post"] = ((dn * on).sum(0), (dn_mag * on.abs()).sum(0))
        else:
            out["do"] = (t, t_mag)
        if gate is not None:
            d, d_mag = dx * m * on * w, mag * m.abs() * (on * w).abs()
            # act' is a difference from 1: its absolute error is a few 2^-24 however small it is
            out["dgate"] = (d.view(G, -1, C).sum(1) * s, d_mag.view(G, -1, C).sum(1) * s.abs().clamp(min=0.05))
    return out
