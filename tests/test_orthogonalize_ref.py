"""The judgement of orthogonalised updates' results accepts the operator's own number formats
and rejects coarser ones and lost terms, rows or tiles (no GPU: mistakes are planted in
the restated formats)."""
import pytest
import torch

import _orth_ref as R

COEFFS = (3.4445, -4.7750, 2.0315)
BF, HF = torch.bfloat16, torch.float16


def gradient(rows, cols, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = max(1, min(rows, cols) // 4)
    left = torch.randn(rows, r, generator=gen) * torch.arange(1, r + 1) ** -0.5
    return (left @ torch.randn(r, cols, generator=gen) + 0.5 * torch.randn(rows, cols, generator=gen)) * 1e-3


class AllBf16(R.Formats):
    low_part = False

    def operand(self, t):
        return t.float().bfloat16().double()


class NoLowPart(R.Formats):
    low_part = False


class OnePass(R.Formats):
    def passes(self, step, m, steps, out_dtype):
        return 1


class OtherCoefficient(R.Formats):
    def poly(self, step, coeffs):
        a, b, c = coeffs
        return a, b * 1.005, c


class NoSquareAtFirst(R.Formats):
    def poly(self, step, coeffs):
        a, b, c = coeffs
        return a, b, 0.0 if step == 0 else c


class NoLowOfGram(R.Formats):
    def rest(self, t, passes):
        return super().rest(t, 1)


def result(g, dt, formats, steps=5):
    shared = R.shares_first_steps(1, *g.shape, steps, dt)
    return R.held(g, steps, COEFFS, 1e-7, 1.0, dt, shared, formats).to(dt)


SHAPES = [(8, 8), (31, 33), (64, 64), (65, 130), (200, 72), (128, 512), (256, 256), (300, 1000), (520, 1032), (1031, 519), (700, 1200), (520, 4200)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_own_formats_are_accepted(rows, cols, dt):
    for seed in range(3 if rows * cols < 100000 else 1):
        g = gradient(rows, cols, seed)
        assert R.problems(result(g, dt, R.Formats()), g, 5, COEFFS) is None
        # and the exact result, rounded
        assert R.problems(R.exact(g, 5, COEFFS).to(dt), g, 5, COEFFS) is None


@pytest.mark.parametrize("rows,cols", SHAPES[:-1])
@pytest.mark.parametrize("formats", [AllBf16, NoLowPart, OtherCoefficient, NoSquareAtFirst, OnePass, NoLowOfGram])
def test_coarser_formats_and_lost_terms_are_rejected(rows, cols, formats):
    g = gradient(rows, cols)
    assert R.problems(result(g, HF, formats()), g, 5, COEFFS) is not None
    if formats in (AllBf16, OtherCoefficient, NoSquareAtFirst):
        assert R.problems(result(g, BF, formats()), g, 5, COEFFS) is not None


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9)] + SHAPES[:-1])
@pytest.mark.parametrize("dt", [BF, HF])
def test_lost_elements_are_rejected(rows, cols, dt):
    g = gradient(rows, cols)
    whole = R.exact(g, 5, COEFFS).to(dt)
    assert R.problems(torch.zeros_like(whole), g, 5, COEFFS) is not None
    assert R.problems(whole.T.contiguous().T * 1.02, g, 5, COEFFS) is not None
    if rows < 8:
        return
    row, tile, ragged = whole.clone(), whole.clone(), whole.clone()
    row[rows // 2] = 0
    tile[:8, :8] = 0
    ragged[rows - 1:, cols - min(cols, 16):] = 0
    for lost in (row, tile, ragged):
        assert R.problems(lost, g, 5, COEFFS) is not None
    other = whole.clone()
    other[0], other[1] = whole[1], whole[0]
    assert R.problems(other, g, 5, COEFFS) is not None


@pytest.mark.parametrize("rows,cols", [(40, 400), (512, 1024), (700, 1200)])
def test_strong_directions(rows, cols):
    """Beside them little is left: the formats' own errors are larger, and still the mistakes show."""
    gen = torch.Generator().manual_seed(1)
    for g in (1 + 0.01 * torch.randn(rows, cols, generator=gen), torch.randn(rows, 1, generator=gen) @ torch.randn(1, cols, generator=gen)
              + 0.005 * torch.randn(rows, cols, generator=gen)):
        for dt in (BF, HF):
            assert R.problems(result(g, dt, R.Formats()), g, 5, COEFFS) is None
        for mistake in (AllBf16, NoLowPart, NoSquareAtFirst, OtherCoefficient, OnePass):
            assert R.problems(result(g, HF, mistake()), g, 5, COEFFS) is not None, mistake
