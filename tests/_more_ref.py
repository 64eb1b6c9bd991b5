"""Definitions in 64 bits of layer norm, of the orthogonalised updates and of the
MoE layer for a few tokens, with what the number formats allow their results to
be off by (EVAL, UNIT and assert_within as in _block_ref)."""
from __future__ import annotations

import math

import torch

from _block_ref import UNIT, product_bound


# ---------------------------------------------------------------- layer norm
def ref_layer_norm(x, w, b, add, eps):
    """{name: (value, sum of its terms' absolute values)}.  A distance from the mean is
    off by a few roundings of |s| + |mean|, and the row's rstd by their ratio to its
    deviation."""
    s = x.double() if add is None else x.double() + add.double()
    mag_s = x.double().abs() if add is None else x.double().abs() + add.double().abs()
    mean = s.mean(1, keepdim=True)
    rstd = ((s - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    far = mag_s.mean(1, keepdim=True)  # what the mean's terms add up to
    wv = 1.0 if w is None else w.double()
    bv = torch.zeros(x.shape[1], dtype=torch.float64, device=x.device) if b is None else b.double()
    n = (s - mean) * rstd
    mag_rstd = rstd * (1 + far * rstd)
    mag_n = rstd * (mag_s + far) + n.abs() * (1 + far * rstd)
    wa = 1.0 if w is None else wv.abs()
    return {"h": (n * wv + bv, mag_n * wa + bv.abs()), "sum": (s, mag_s), "mean": (mean[:, 0], far[:, 0]),
            "rstd": (rstd[:, 0], mag_rstd[:, 0])}


def ref_layer_norm_bwd(dh, s, mean, rstd, w, dsum):
    dh, s, mean, rstd = dh.double(), s.double(), mean.double()[:, None], rstd.double()[:, None]
    wv = torch.ones(s.shape[1], dtype=torch.float64, device=s.device) if w is None else w.double()
    d = 0.0 if dsum is None else dsum.double()
    n, big = (s - mean) * rstd, (s.abs() + mean.abs()) * rstd  # n is off by roundings of `big`
    g = dh * wv
    dx = d + rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    mag = (0.0 if dsum is None else d.abs()) + rstd * (g.abs() + g.abs().mean(1, keepdim=True) + big * (g.abs() * big).mean(1, keepdim=True))
    return {"dx": (dx, mag), "dw": ((dh * n).sum(0), (dh.abs() * big).sum(0)), "db": (dh.sum(0), dh.abs().sum(0))}


# ---------------------------------------------------------------- orthogonalised updates
def ref_orthogonalize(g, steps, coeffs, eps, scale, out_dtype):
    """(X, what its Frobenius norm may be off by) of one matrix.

    The products' operands are fp16: the rounding of an entry v is uniform within
    u |v| or less, u = 2^-11, so its root mean square is at most u |v| / sqrt(3), and
    of E with such independent entries |E M|_F^2 has the mean sum_ij r_ij^2 |M_j|^2.
    First order, the roundings of one step:
      X (in B X and in the Gram matrix), A and B off their diagonals;
    a step takes an error of its input to the next by at most the largest slope of
    its polynomial on [0, largest singular value].  Of the sum, four times is allowed
    (a Frobenius norm of thousands of terms keeps close to its mean; the smallest
    matrices' few do not), and 2^-24's accumulation over the products' length."""
    a, b, c = coeffs
    u = 2.0 ** -11 / math.sqrt(3)
    x = g.double()
    x = x if x.shape[0] <= x.shape[1] else x.T
    norm = torch.linalg.vector_norm(x) + eps
    x = x / norm if float(norm) > 0 else x
    err = torch.zeros((), dtype=torch.float64, device=g.device)
    sigma = torch.linalg.svdvals(x)  # they go through the polynomial one by one
    for _ in range(steps):
        gram = x @ x.T
        poly = b * gram + c * gram @ gram
        off = lambda t: t - torch.diag(torch.diagonal(t))
        top = sigma.abs().max()
        sq = x.square()
        rms = lambda e2, m2: u * torch.sqrt((e2 * m2).sum())  # entries' squares, squared row norms of the other factor
        gain = (abs(b) + 2 * abs(c) * top ** 2)
        eta = rms(sq.sum(1), off(poly).square().sum(0))  # B_off E
        eta = eta + gain * top * 2 * rms(sq, x.square().sum(0)[None, :])  # (E X^T + X E^T) through the polynomial
        eta = eta + gain * rms(off(gram).square(), sq.sum(1)[None, :]) + rms(off(poly).square(), sq.sum(1)[None, :])
        eta = eta + product_bound(max(x.shape)) * (abs(a) + gain * top ** 2 + (b * sigma ** 2 + c * sigma ** 4).abs().max()) * torch.linalg.vector_norm(x)
        s = torch.linspace(0, 1, 257, dtype=torch.float64, device=g.device) * top
        slope = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs().max()
        err = slope * err + eta
        x = a * x + poly @ x
        sigma = a * sigma + b * sigma ** 3 + c * sigma ** 5
    x = scale * (x if g.shape[0] <= g.shape[1] else x.T)
    return x, float(4 * abs(scale) * err + UNIT[out_dtype] * torch.linalg.vector_norm(x) + 1e-30)


# ---------------------------------------------------------------- a few tokens
def ref_route(logits, k):
    """idx, w: NaN ranks below all numbers, a chosen -inf weighs 0."""
    idx, w = [], []
    for row in logits.double().tolist():
        order = sorted(range(len(row)), key=lambda e: (row[e] != row[e], -row[e] if row[e] == row[e] else 0.0, e))[:k]
        top = row[order[0]]
        z = [0.0 if row[e] == -math.inf else (math.nan if not math.isfinite(top) or row[e] != row[e] else math.exp(row[e] - top)) for e in order]
        t = sum(z)
        idx.append(order)
        w.append([0.0 if row[e] == -math.inf else (v / t) for e, v in zip(order, z)])
    return idx, w


def ref_few_tokens(x, wg, wu, wd, idx, w, dead):
    """out and its bound.  dead: pairs without a part.  h is held in two numbers of
    the type: off by UNIT^2 of itself (and, in fp16, by half the smallest subnormal)."""
    x64, T, (H, I) = x.double(), x.shape[0], wd.shape[1:]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    bound = torch.zeros_like(out)
    up, down = product_bound(H), product_bound(2 * I)
    held = UNIT[x.dtype] ** 2
    for t in range(T):
        for j, (e, v) in enumerate(zip(idx[t], w[t])):
            if dead[t][j]:
                continue
            row, a = x64[t], x64[t].abs()
            mg, mu, md = wg[e].double(), wu[e].double(), wd[e].double()
            g, u = mg @ row, mu @ row
            eg, eu = up * (mg.abs() @ a), up * (mu.abs() @ a)
            silu = g * torch.sigmoid(g)
            h = silu * u
            eh = 1.1 * eg * u.abs() + silu.abs() * eu + 1.1 * eg * eu + h.abs() * (held + 3e-6) + 2.0 ** -25
            out[t] += v * (md @ h)
            bound[t] += v * (md.abs() @ (eh + down * h.abs())) * 1.0001 + 4e-6 * v * (md.abs() @ h.abs())
    return out, bound + UNIT[x.dtype] * out.abs() + 2.0 ** -25
