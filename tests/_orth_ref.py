"""Orthogonalised updates in 64 bits: the definition, and the definition with the roundings
of the formats that the operator states (X as two fp16 numbers, Gram matrices and their
polynomials as a diagonal in fp32 and a rest of one or two fp16 numbers), so that a test
can ask how far those formats, and no others, put a result from the exact one."""
from __future__ import annotations

import math

import torch

from _block_ref import UNIT

X_SCALE, A_SCALE, B_SCALE = 8192.0, 1024.0, 256.0
PRECISE_SIDE, ROUGH_STEPS = 512, 2


def _wide(g):
    return g.double() if g.shape[0] <= g.shape[1] else g.double().T


def exact(g, steps, coeffs, eps=1e-7, scale=1.0):
    a, b, c = coeffs
    x = _wide(g)
    x = x / (torch.linalg.vector_norm(x) + eps)
    for _ in range(steps):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return scale * (x if g.shape[0] <= g.shape[1] else x.T)


def shares_first_steps(count, rows, cols, steps, out_dtype, num_sms=152):
    """Whether the first two steps go through one update."""
    m, n = min(rows, cols), max(rows, cols)
    tm = (m + 255) // 256
    small = tm * (tm + 1) * count <= num_sms // 2
    return passes_of(0, m, steps, out_dtype) == 1 and steps >= 2 and (n >= 8 * m if small else 2 * n >= 3 * m)


def passes_of(step, m, steps, out_dtype):
    return 3 if out_dtype == torch.float16 or (m <= PRECISE_SIDE and step + ROUGH_STEPS < steps) else 1


def _fp32(t):
    return t.float().double()


class Formats:
    """What is rounded to what; the subclasses of the tests plant mistakes here."""
    low_part = True  # of X

    def operand(self, t):
        return t.float().half().double()

    def state(self, x):
        hi = self.operand(x)
        return hi, self.operand(x - hi) if self.low_part else torch.zeros_like(hi)

    def rest(self, t, passes):  # a symmetric matrix without its diagonal
        t = t - torch.diag(torch.diagonal(t))
        hi = self.operand(t)
        return hi, self.operand(t - hi) if passes > 1 else torch.zeros_like(hi)

    def passes(self, step, m, steps, out_dtype):
        return passes_of(step, m, steps, out_dtype)

    def product(self, x, y, passes):
        s = x[0] @ y[0]
        return s + x[0] @ y[1] + x[1] @ y[0] if passes > 1 else s

    def poly(self, step, coeffs):
        return coeffs


def held(g, steps, coeffs, eps, scale, out_dtype, shared, formats=Formats()):
    """The result before its rounding, with exact sums."""
    f, P = formats, formats.product
    x = _wide(g)
    m = x.shape[0]
    norm = torch.linalg.vector_norm(x) + eps
    x = f.state(_fp32(x * (X_SCALE / norm)))
    value = x[0] + x[1]
    i = 0

    def symmetric(y, diag, passes):
        return _fp32(diag), f.rest(_fp32(y), passes)

    def polynomial(d, o, b, c, passes):
        s = P(o, o, passes) * (B_SCALE / A_SCALE ** 2)
        y = (b + c * (d[:, None] + d[None, :])) * ((o[0] + o[1]) * (B_SCALE / A_SCALE)) + c * s
        return symmetric(y, d * (b + c * d) + c * torch.diagonal(s) / B_SCALE, passes)

    def mixed(d1, o1, s1, a1, d2, o2, a2, to):
        s = P(o1, o2, 1) * (to / (s1 * B_SCALE))
        y = (d1 + a1)[:, None] * (o2[0] * (to / B_SCALE)) + (d2 + a2)[None, :] * (o1[0] * (to / s1)) + s
        return symmetric(y, (d1 + a1) * (d2 + a2) + torch.diagonal(s) / to, 1)

    while i < steps:
        a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in f.poly(i, coeffs))
        passes = f.passes(i, m, steps, out_dtype)
        gram = P(x, (x[0].T, x[1].T), passes) * (A_SCALE / X_SCALE ** 2)
        d, o = symmetric(gram, torch.diagonal(gram) / A_SCALE, passes)
        e, q = polynomial(d, o, b, c, passes)
        shift = a
        if shared and i == 0:
            wd, w = mixed(d, o, A_SCALE, 0.0, e, q, a, A_SCALE)
            d, o = mixed(wd, w, A_SCALE, 0.0, e, q, a, A_SCALE)
            e2, q2 = polynomial(d, o, b, c, passes)
            e, q = mixed(e2, q2, B_SCALE, a, e, q, a, B_SCALE)
            shift, i = 0.0, 1
        i += 1
        value = _fp32((shift + e)[:, None] * (x[0] + x[1]) + P(q, x, passes) / B_SCALE)
        x = f.state(value)
    value = value * (scale / X_SCALE)
    return value if g.shape[0] <= g.shape[1] else value.T


def sums_error(g, steps, coeffs, eps, scale):
    """What the accumulators leave: they drop what is below their last bit at every 16 of a
    product's length, half a unit of 2^-23 on average and always to one side, so a Gram
    matrix is off by about K / 16 * 2^-24 of itself, and so is B X.  Each singular value s goes through
    the polynomial by itself: its error through the slope, the Gram matrix' through b s^3 +
    2 c s^5.  Twice that is allowed."""
    a, b, c = coeffs
    x = _wide(g)
    m, n = x.shape
    s = torch.linalg.svdvals(x / (torch.linalg.vector_norm(x) + eps))
    long, short = (n / 16 + 8) * 2.0 ** -24, (m / 16 + 8) * 2.0 ** -24
    err = torch.zeros_like(s)
    for _ in range(steps):
        err = ((a + 3 * b * s ** 2 + 5 * c * s ** 4).abs() * err + (b * s ** 3 + 2 * c * s ** 5).abs() * long
               + (b * s ** 3 + c * s ** 5).abs() * short)
        s = a * s + b * s ** 3 + c * s ** 5
    return 2 * abs(scale) * float(torch.linalg.vector_norm(err))


def problems(out, g, steps, coeffs, eps=1e-7, scale=1.0, count=1):
    """What is wrong with a result, or None.

    Its norm's distance from the exact one: the formats' (held, half as much again), the sums' and
    its own rounding, which have nothing to do with one another, so their squares add up; a
    sum of N rounding errors' squares keeps within 3 / sqrt(N) of what is expected.  And in
    every tile of 32 x 32 (where a lost row or tile would not show in the norm of all) a
    twentieth of what a tile holds on average and of what this one holds."""
    dt = out.dtype
    ref = exact(g, steps, coeffs, eps, scale)
    formats = held(g, steps, coeffs, eps, scale, dt, shares_first_steps(count, *g.shape, steps, dt))
    norm, dist = float(torch.linalg.vector_norm(ref)), float(torch.linalg.vector_norm(formats - ref))
    spread = 3 / math.sqrt(g.numel())
    # (the rounding of few elements can happen to be small: at least half of a rounding's mean square, u^2 / 6)
    rounding = max(float(torch.linalg.vector_norm(ref.to(dt).double() - ref)), min(1.0, spread) * UNIT[dt] * norm / math.sqrt(6))
    allowed = math.sqrt(rounding ** 2 + (1.5 * dist) ** 2 + sums_error(g, steps, coeffs, eps, scale) ** 2) * (1 + spread) + 1e-30
    diff = out.double() - ref
    err = float(torch.linalg.vector_norm(diff))
    if not err <= allowed:
        return f"off by {err / norm:.2e} of the norm, {allowed / norm:.2e} allowed (rounding {rounding / norm:.2e}, formats {dist / norm:.2e})"

    def tiles(t):
        r, c = (-(-k // 32) * 32 for k in t.shape)
        p = torch.zeros(r, c, dtype=torch.float64, device=t.device)
        p[:t.shape[0], :t.shape[1]] = t.square()
        return p.view(r // 32, 32, c // 32, 32).sum((1, 3)).sqrt()

    full = tiles(torch.ones_like(ref))  # the root of a tile's elements
    lost = tiles(diff) > 0.05 * (full * (norm / math.sqrt(ref.numel())) + tiles(ref)) + 1e-30
    return f"{int(lost.sum())} tiles off, the first {lost.nonzero()[0].tolist()}" if bool(lost.any()) else None
