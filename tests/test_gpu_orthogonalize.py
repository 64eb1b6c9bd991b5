"""Orthogonalised updates against the definition in 64 bits."""
import ctypes

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _more_ref import ref_orthogonalize

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)


def work_for(count, rows, cols, least=False):
    return torch.empty(sm.moe_orthogonalize_workspace(count, rows, cols, least), dtype=torch.uint8, device="cuda").fill_(255)


def gradient(count, rows, cols, dt=torch.bfloat16, seed=0, scale=1e-3):
    gen = torch.Generator("cuda").manual_seed(seed)
    r = max(1, min(rows, cols) // 4)
    left = torch.randn(count, rows, r, generator=gen, device="cuda") * torch.arange(1, r + 1, device="cuda") ** -0.5
    g = left @ torch.randn(count, r, cols, generator=gen, device="cuda") + 0.5 * torch.randn(count, rows, cols, generator=gen, device="cuda")
    return (g * scale).to(dt)


def check(g, out, steps=5, coeffs=COEFFS, eps=1e-7, scale=1.0):
    for i in range(g.shape[0]):
        ref, bound = ref_orthogonalize(g[i], steps, coeffs, eps, scale, out.dtype)
        err = float(torch.linalg.vector_norm(out[i].double() - ref))
        assert err <= bound, (i, tuple(g.shape), err, bound, float(torch.linalg.vector_norm(ref)))


SIZES = [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 8, 8), (1, 31, 33), (2, 64, 64), (2, 65, 130), (1, 200, 72), (3, 128, 512),
         (2, 256, 256), (1, 257, 255), (2, 300, 1000), (1, 1031, 519), (1, 520, 1032), (1, 640, 2049), (30, 72, 136),
         (1, 72, 4100), (2, 4100, 72), (1, 300, 2100), (1, 2100, 500), (3, 1300, 1288),
         (1, 33000, 40), (1, 24, 20000)]


@pytest.mark.parametrize("count,rows,cols", SIZES)
@pytest.mark.parametrize("dt,out_dt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                       (torch.float32, torch.bfloat16), (torch.float32, torch.float16)])
def test_sizes(count, rows, cols, dt, out_dt):
    g = gradient(count, rows, cols, dt, scale=1e-1 if dt == torch.float16 else 1e-3)
    out = torch.empty(count, rows, cols, device="cuda", dtype=out_dt)
    sm.moe_orthogonalize(g, out, work_for(count, rows, cols))
    check(g, out)


@pytest.mark.parametrize("rows,cols", [(129, 300), (300, 129)])
@pytest.mark.parametrize("steps,coeffs", [(0, COEFFS), (1, COEFFS), (2, (1.5, -0.5, 0.0)), (3, (1.875, -1.25, 0.375)), (12, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(rows, cols, steps, coeffs):
    g = gradient(2, rows, cols, torch.float32)
    out = torch.empty(2, rows, cols, device="cuda", dtype=torch.float16)
    sm.moe_orthogonalize(g, out, work_for(2, rows, cols), steps=steps, coeffs=coeffs, scale=-0.25)
    check(g, out, steps, coeffs, scale=-0.25)


@pytest.mark.parametrize("count,rows,cols", [(40, 72, 136), (40, 136, 72), (8, 600, 1000), (8, 1000, 600), (1, 40, 400), (2, 700, 64)])
@pytest.mark.parametrize("out_dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("steps", [2, 5, 6])
def test_first_two_steps_with_one_update(count, rows, cols, out_dt, steps):
    """Shapes whose first two steps go through one update."""
    g = gradient(count, rows, cols, torch.float32)
    out = torch.empty(count, rows, cols, device="cuda", dtype=out_dt)
    sm.moe_orthogonalize(g, out, work_for(count, rows, cols), steps=steps)
    check(g[:3], out[:3], steps)


@pytest.mark.parametrize("rows,cols", [(64, 200), (200, 64), (300, 300), (16, 300)])
def test_orthogonal_rows_take_the_scalar_recursion(rows, cols):
    """One entry in each row and column: every Gram matrix is diagonal, held in 32
    bits, and the entries go through the polynomial one by one."""
    m = min(rows, cols)
    gen = torch.Generator("cuda").manual_seed(3)
    v = torch.randn(m, generator=gen, device="cuda")
    g = torch.zeros(1, rows, cols, device="cuda")
    at_r, at_c = torch.randperm(rows, generator=gen, device="cuda")[:m], torch.randperm(cols, generator=gen, device="cuda")[:m]
    g[0, at_r, at_c] = v
    out = torch.empty(1, rows, cols, device="cuda", dtype=torch.float16)
    sm.moe_orthogonalize(g, out, work_for(1, rows, cols))
    x = v.double() / (torch.linalg.vector_norm(v.double()) + 1e-7)
    (a, b, c), err = COEFFS, torch.zeros_like(x)
    for _ in range(5):
        # The Gram matrix' operands are x to 2^-11, so its diagonal x^2 is off by 2 * 2^-11
        # + 2^-22 of itself, and B's b x^2 + c x^4 by (b x^2 + 2 c x^4) times that; x itself
        # is held to 2^-22 (or 2^-25 / 2^13 of one); the rest is fp32's.
        off = 2 * 2.0 ** -11 + 2.0 ** -22
        err = ((a + 3 * b * x ** 2 + 5 * c * x ** 4).abs() * err + off * (1 + off) * (x * (b * x ** 2 + 2 * c * x ** 4)).abs()
               + off * off * (c * x ** 5).abs() + 1e-6 * x.abs() * (abs(a) + abs(b) * x ** 2 + c * x ** 4) + 1e-8)
        x = a * x + b * x ** 3 + c * x ** 5
    got = out[0, at_r, at_c].double()
    assert bool(((got - x).abs() <= 2.0 ** -11 * x.abs() + 1.01 * err).all())
    rest = out[0].clone()
    rest[at_r, at_c] = 0
    assert not rest.any()


@pytest.mark.parametrize("dt,size", [(torch.float32, 1e30), (torch.float32, 1e-25), (torch.bfloat16, 1e35), (torch.float16, 1e3)])
def test_range(dt, size):
    """The norm's squares beyond the range of 32 bits; eps 0, so that the scale does not matter."""
    g = gradient(2, 96, 160, torch.float32, scale=size).to(dt)
    out = torch.empty(2, 96, 160, device="cuda", dtype=torch.bfloat16)
    sm.moe_orthogonalize(g, out, work_for(2, 96, 160), eps=0.0)
    check(g, out, eps=0.0)


@pytest.mark.parametrize("rows,cols", [(100, 300), (300, 100)])
def test_one_matrix_does_not_touch_another(rows, cols):
    g = gradient(5, rows, cols)
    want = torch.empty_like(g)
    sm.moe_orthogonalize(g, want, work_for(5, rows, cols))
    g[1] = 0
    g[2, rows // 2, 3] = float("nan")
    g[4, 0, 0] = float("inf")
    out = torch.empty_like(g)
    sm.moe_orthogonalize(g, out, work_for(5, rows, cols))
    assert not out[1].any() and bool(out[2].isnan().all()) and bool(out[4].isnan().all())
    assert torch.equal(out[0], want[0]) and torch.equal(out[3], want[3])


@pytest.mark.parametrize("rows,cols", [(72, 250), (250, 72), (64, 64)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_strides_and_turns(rows, cols, dt):
    """Rows and matrices apart, off every alignment; the least workspace takes the
    matrices one at a time, with the same results."""
    count, ld, stride = 4, cols + 5, (cols + 5) * (rows + 2) + 3
    flat = torch.zeros(stride * count + 1, device="cuda", dtype=dt)
    g = flat[1:].as_strided((count, rows, cols), (stride, ld, 1))
    g.copy_(gradient(count, rows, cols, dt))
    plain = torch.empty(count, rows, cols, device="cuda", dtype=torch.bfloat16)
    sm.moe_orthogonalize(g.contiguous(), plain, work_for(count, rows, cols))
    buf = torch.full((stride * count + 1,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = buf[1:].as_strided((count, rows, cols), (stride, ld, 1))
    for least in (False, True):
        out.fill_(1)
        sm.moe_orthogonalize(g, out, work_for(count, rows, cols, least))
        assert torch.equal(out, plain)
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask[1:].as_strided((count, rows, cols), (stride, ld, 1)).fill_(False)
    assert bool((buf[mask] == 7).all())


def test_two_dimensions_and_in_place():
    g = gradient(1, 130, 70)
    want = torch.empty_like(g)
    work = work_for(1, 130, 70)
    sm.moe_orthogonalize(g, want, work)
    one = g[0].clone()
    sm.moe_orthogonalize(one, one, work)
    assert torch.equal(one, want[0])


def test_capture_and_streams():
    g = gradient(3, 200, 400)
    out, work = torch.empty_like(g), work_for(3, 200, 400)
    sm.moe_orthogonalize(g, out, work)
    want = out.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sm.moe_orthogonalize(g, out, work)
        with torch.cuda.graph(graph, stream=side):
            sm.moe_orthogonalize(g, out, work)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        out.zero_()
        work.fill_(255)
        graph.replay()
        assert torch.equal(out, want)


def test_no_matrices():
    e = torch.empty(0, 8, 8, device="cuda", dtype=torch.bfloat16)
    sm.moe_orthogonalize(e, e, torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_refusals():
    g = gradient(2, 40, 72)
    out, work = torch.empty_like(g), work_for(2, 40, 72)
    bad = [lambda: sm.moe_orthogonalize(g, out[:1], work), lambda: sm.moe_orthogonalize(g, out.float(), work),
           lambda: sm.moe_orthogonalize(g.cpu(), out, work), lambda: sm.moe_orthogonalize(g, out, work.cpu()),
           lambda: sm.moe_orthogonalize(g.transpose(1, 2), out.transpose(1, 2), work), lambda: sm.moe_orthogonalize(g[0, 0], out[0, 0], work),
           lambda: sm.moe_orthogonalize(g, out, work, steps=65), lambda: sm.moe_orthogonalize(g, out, work, steps=-1),
           lambda: sm.moe_orthogonalize(g, out, work, eps=-1.0), lambda: sm.moe_orthogonalize(g, out, work, coeffs=(1.0, 2.0)),
           lambda: sm.moe_orthogonalize(g, out, work[128:]), lambda: sm.moe_orthogonalize(g, out, work, status=out),
           lambda: sm.moe_orthogonalize(g[:1].expand(2, 40, 72), out, work), lambda: sm.moe_orthogonalize(g, out[:1].expand(2, 40, 72), work)]
    for i, call in enumerate(bad):
        with pytest.raises(sm.SymmoeError) as e:
            call()
        assert e.value.code == sm.SYM_EINVAL, i
    least = sm.moe_orthogonalize_workspace(2, 40, 72, least=True)
    with pytest.raises(sm.SymmoeError) as e:
        sm.moe_orthogonalize(g, out, work[:least - 256])
    assert e.value.code == sm.SYM_ENOSPACE


def test_workspace_fills_the_device_and_no_more():
    """Many large matrices go through in turns; few or small ones side by side."""
    one = sm.moe_orthogonalize_workspace(256, 2048, 7168, least=True)
    assert one == sm.moe_orthogonalize_workspace(1, 2048, 7168)
    assert sm.moe_orthogonalize_workspace(8, 2048, 7168) == 8 * one
    assert sm.moe_orthogonalize_workspace(256, 2048, 7168) < 4 << 30
    small = sm.moe_orthogonalize_workspace(1, 64, 64)
    assert sm.moe_orthogonalize_workspace(100, 64, 64) == 100 * small


def test_a_wait_that_runs_out_is_reported():
    """Waits limited to 20 us where a tile's K axis takes about a millisecond (the limit is
    looked at every sixteenth poll, and a poll can take some microseconds): the kernels
    give up, say so, and leave the device as they found it."""
    rows, cols = 600, 65536
    g = gradient(1, rows, cols, torch.float16, scale=1e-1)
    out, work, status = torch.empty_like(g), work_for(1, rows, cols), torch.zeros(1, dtype=torch.int32, device="cuda")
    sm.moe_orthogonalize(g, out, work, status=status)
    want = out.clone()
    assert int(status) == 0
    a = sm.SymOrthogonalize(1, rows, cols, 1, sm.SYM_FP16, sm.SYM_FP16, (ctypes.c_float * 3)(*COEFFS), 1e-7, 1.0, 20,
                            status.data_ptr(), g.data_ptr(), out.data_ptr(), rows * cols, cols, rows * cols, cols, work.data_ptr(),
                            work.numel())
    assert sm.lib().moe_orthogonalize(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == sm.SYM_OK
    torch.cuda.synchronize()
    assert int(status) & sm.SYM_STATUS_TIMEOUT
    status.zero_()
    out.zero_()
    sm.moe_orthogonalize(g, out, work, status=status)
    assert int(status) == 0 and torch.equal(out, want)
