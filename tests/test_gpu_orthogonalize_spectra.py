"""Orthogonalised updates of gradients with strong directions, against the definition
in 64 bits: the errors that the interface promises, whatever the spectrum."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
COEFFS = (3.4445, -4.7750, 2.0315)


def with_values(rows, cols, s, gen):
    """A matrix of these singular values (for the shorter side)."""
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float64)
    m, n = min(rows, cols), max(rows, cols)
    left, right = torch.linalg.qr(rand(m, m))[0], torch.linalg.qr(rand(n, m))[0]
    g = (left * s) @ right.T
    return g if rows <= cols else g.T


def gradient(kind, rows, cols, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float64)
    m = min(rows, cols)
    i = torch.arange(1, m + 1, device="cuda", dtype=torch.float64)
    some = lambda k, rest: torch.where(i <= k, 1.0, rest)
    return {"broad": lambda: rand(rows, cols),
            "inverse": lambda: with_values(rows, cols, 1 / i, gen),
            "inverse squares": lambda: with_values(rows, cols, i ** -2, gen),
            "mean": lambda: 3 + rand(rows, cols),
            "mean and little": lambda: 1 + 0.01 * rand(rows, cols),
            "one and 1e-2": lambda: with_values(rows, cols, some(1, 1e-2), gen),
            "eight and 1e-3": lambda: with_values(rows, cols, some(8, 1e-3), gen),
            "one and 1e-4": lambda: with_values(rows, cols, some(1, 1e-4), gen),
            "one and noise": lambda: rand(rows, 1) @ rand(1, cols) + 0.005 * rand(rows, cols),
            "rank one": lambda: rand(rows, 1) @ rand(1, cols),
            "rank eight": lambda: rand(rows, 8) @ rand(8, cols)}[kind]().float().contiguous()


ALONE = ("eight and 1e-3", "one and 1e-4", "rank one", "rank eight")  # a few directions with next to nothing beside them


def exact(g, steps=5):
    """X of one matrix, in 64 bits."""
    a, b, c = COEFFS
    x = g.double() if g.shape[0] <= g.shape[1] else g.double().T
    x = x / (torch.linalg.vector_norm(x) + 1e-7)
    for _ in range(steps):
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x if g.shape[0] <= g.shape[1] else x.T


def promised(kind, rows, cols, dt):
    if dt == HF:
        return 6e-4 if kind in ALONE else 2e-4
    return 2e-3 if min(rows, cols) < 16 else 1.2e-3


def check(kind, g, out):
    """Off by what is promised and by the result's rounding, which are independent of one another:
    their squares add up, to 3 / sqrt(elements) of the sum (three deviations of a sum of
    so many independent terms)."""
    ref = exact(g)
    norm = float(torch.linalg.vector_norm(ref))
    rounding = float(torch.linalg.vector_norm(ref.to(out.dtype).double() - ref))
    err = float(torch.linalg.vector_norm(out.double() - ref))
    allowed = (rounding ** 2 + (promised(kind, *g.shape, out.dtype) * norm) ** 2) ** 0.5 * (1 + 3 / g.numel() ** 0.5)
    assert err <= allowed, (kind, tuple(g.shape), err / norm, rounding / norm, allowed / norm)


KINDS = ["broad", "inverse", "inverse squares", "mean", "mean and little", "one and 1e-2", "eight and 1e-3", "one and 1e-4",
         "one and noise", "rank one", "rank eight"]
# both sides of the products' precision rule, sizes that share the first two steps, wide and tall
SHAPES = [(8, 8), (40, 400), (64, 700), (256, 2048), (2048, 256), (512, 1024), (513, 600), (600, 1000), (1000, 600), (520, 4400)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("out_dt", [BF, HF])
def test_error_is_what_is_promised(kind, rows, cols, out_dt):
    g = gradient(kind, rows, cols)
    out = torch.empty(rows, cols, device="cuda", dtype=out_dt)
    sm.moe_orthogonalize(g, out, torch.empty(sm.moe_orthogonalize_workspace(1, rows, cols), dtype=torch.uint8, device="cuda"))
    check(kind, g, out)


@pytest.mark.parametrize("kind", ["broad", "mean and little", "eight and 1e-3", "rank one"])
@pytest.mark.parametrize("count,rows,cols", [(5, 1031, 519), (3, 2048, 7168)])
@pytest.mark.parametrize("out_dt", [BF, HF])
def test_batches(kind, count, rows, cols, out_dt):
    g = torch.stack([gradient(kind, rows, cols, seed) for seed in range(count)])
    out = torch.empty(count, rows, cols, device="cuda", dtype=out_dt)
    sm.moe_orthogonalize(g, out, torch.empty(sm.moe_orthogonalize_workspace(count, rows, cols), dtype=torch.uint8, device="cuda"))
    for i in (0, count - 1):
        check(kind, g[i], out[i])
