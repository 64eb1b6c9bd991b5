"""Orthogonalised updates against the definition in 64 bits, no further from it than the
operator's number formats put them, and no tile of 32 x 32 lost."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _orth_ref import problems, shares_first_steps

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
COEFFS = (3.4445, -4.7750, 2.0315)


def gradient(count, rows, cols, dt=torch.float32, seed=0, scale=1e-3):
    """Strong directions over a broad rest."""
    gen = torch.Generator("cuda").manual_seed(seed)
    r = max(1, min(rows, cols) // 4)
    left = torch.randn(count, rows, r, generator=gen, device="cuda") * torch.arange(1, r + 1, device="cuda") ** -0.5
    g = left @ torch.randn(count, r, cols, generator=gen, device="cuda") + 0.5 * torch.randn(count, rows, cols, generator=gen, device="cuda")
    return (g * scale).to(dt)


def run(g, out_dt, **kw):
    work = torch.empty(sm.moe_orthogonalize_workspace(*g.shape), dtype=torch.uint8, device="cuda").fill_(255)
    out = torch.full(g.shape, 7.0, device="cuda", dtype=out_dt)
    sm.moe_orthogonalize(g, out, work, **kw)
    return out


def check(g, out, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0):
    for i in sorted({0, g.shape[0] // 2, g.shape[0] - 1}):
        wrong = problems(out[i], g[i], steps, coeffs, eps, scale, g.shape[0])
        assert wrong is None, (i, wrong)


# one matrix and batches, tiles that end inside, products of one tile and of many, a long K axis in parts
SIZES = [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 8, 8), (1, 31, 33), (2, 64, 64), (2, 65, 130), (1, 200, 72), (3, 128, 512),
         (2, 256, 256), (1, 257, 255), (2, 300, 1000), (1, 1031, 519), (1, 520, 1032), (1, 640, 2049), (30, 72, 136),
         (1, 72, 4100), (2, 4100, 72), (1, 300, 2100), (1, 2100, 500), (3, 1300, 1288), (1, 24, 20000)]


@pytest.mark.parametrize("count,rows,cols", SIZES)
@pytest.mark.parametrize("dt,out_dt", [(BF, BF), (HF, HF), (torch.float32, BF), (torch.float32, HF)])
def test_sizes(count, rows, cols, dt, out_dt):
    g = gradient(count, rows, cols, dt, scale=1e-1 if dt == HF else 1e-3)
    check(g, run(g, out_dt))


@pytest.mark.parametrize("count,rows,cols,steps", [(8, 600, 1000, 5), (8, 1000, 600, 5), (1, 520, 4200, 5), (1, 4200, 520, 6), (3, 700, 6000, 2),
                                                   (40, 136, 72, 2), (2, 700, 64, 2), (8, 800, 1300, 3)])
def test_first_two_steps_with_one_update(count, rows, cols, steps):
    assert shares_first_steps(count, rows, cols, steps, BF)
    g = gradient(count, rows, cols)
    check(g, run(g, BF, steps=steps), steps)


@pytest.mark.parametrize("rows,cols", [(129, 300), (300, 129), (600, 700)])
@pytest.mark.parametrize("out_dt", [BF, HF])
@pytest.mark.parametrize("steps,coeffs", [(0, COEFFS), (1, COEFFS), (2, (1.5, -0.5, 0.0)), (3, (1.875, -1.25, 0.375)), (8, (1.5, -0.5, 0.0)),
                                          (8, COEFFS)])
def test_steps_and_coefficients(rows, cols, out_dt, steps, coeffs):
    g = gradient(2, rows, cols)
    check(g, run(g, out_dt, steps=steps, coeffs=coeffs, scale=-0.25), steps, coeffs, scale=-0.25)


@pytest.mark.parametrize("count,rows,cols,out_dt", [(1, 2048, 7168, HF), (1, 7168, 2048, BF)])
def test_large(count, rows, cols, out_dt):
    g = gradient(count, rows, cols)
    check(g, run(g, out_dt))
