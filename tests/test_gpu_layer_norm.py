"""Layer norm and its gradient against their definitions in 64 bits."""
import itertools

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import assert_within
from _more_ref import ref_layer_norm, ref_layer_norm_bwd

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(rows, cols, dt, pad=0, shift=0, far=0.0, seed=0):
    """[rows, cols] with a row stride of cols + pad, starting `shift` elements in; rows around `far`."""
    gen = torch.Generator("cuda").manual_seed(seed)
    ld = cols + pad
    flat = torch.randn(rows * ld + shift, generator=gen, device="cuda") + far
    return flat.to(dt)[shift:].as_strided((rows, cols), (ld, 1))


def like(t):
    """An output of the same layout; what no row covers holds a pattern."""
    n = t.untyped_storage().size() // t.element_size()
    return torch.full((n,), 77.0, device="cuda", dtype=t.dtype).as_strided(t.shape, t.stride(), t.storage_offset())


def untouched(t):
    flat = torch.as_strided(t, (t.untyped_storage().size() // t.element_size(),), (1,), 0)
    mask = torch.ones_like(flat, dtype=torch.bool)
    torch.as_strided(mask, t.shape, t.stride(), t.storage_offset()).fill_(False)
    return bool((flat[mask] == 77).all())


SIZES = [(1, 1), (3, 1), (1, 7), (5, 8), (2, 31), (4, 129), (3, 1000), (2, 1001), (7, 4096), (3, 7168), (2, 8192), (2, 8193),
         (2, 16384), (3, 20001), (1, 65536), (700, 264), (1300, 96), (33, 4104)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", TYPES)
def test_forward(rows, cols, dt):
    x, add, w, b = make(rows, cols, dt, far=0.5), make(rows, cols, dt, seed=1), make(1, cols, dt, seed=2)[0], make(1, cols, dt, seed=3)[0]
    for with_add, with_w, with_b in itertools.product((False, True), repeat=3):
        h, total = like(x), like(x)
        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        a = add if with_add else None
        sm.moe_layer_norm(x, h, w=w if with_w else None, b=b if with_b else None, add=a, sum=total, mean=mean, rstd=rstd)
        ref = ref_layer_norm(x, w if with_w else None, b if with_b else None, a, 1e-5)
        for name, got in (("h", h), ("sum", total), ("mean", mean), ("rstd", rstd)):
            assert_within(got, *ref[name], name)


@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 8), (0, 1), (3, 5), (16, 2)])
@pytest.mark.parametrize("cols", [40, 520, 1003, 4096, 9000])
@pytest.mark.parametrize("dt", TYPES)
def test_strides(pad, shift, cols, dt):
    x, add = make(9, cols, dt, pad, shift), make(9, cols, dt, 8, 0, seed=1)
    h, total = like(x), like(add)
    w = make(1, cols, dt, 0, shift, seed=2)[0]
    mean, rstd = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    sm.moe_layer_norm(x, h, w=w, add=add, sum=total, mean=mean, rstd=rstd)
    ref = ref_layer_norm(x, w, None, add, 1e-5)
    assert_within(h, *ref["h"], "h")
    assert_within(total, *ref["sum"], "sum")
    assert untouched(h) and untouched(total)
    dh, dsum = make(9, cols, dt, 0, 0, seed=3), make(9, cols, dt, pad, shift, seed=4)
    dx, dw, db = like(x), torch.empty_like(w), torch.empty(cols + 1, device="cuda", dtype=dt)[1:]
    work = torch.empty(sm.moe_layer_norm_workspace(9, cols), dtype=torch.uint8, device="cuda")
    sm.moe_layer_norm_bwd(dh, x, mean, rstd, dx=dx, w=w, dsum=dsum, dw=dw, db=db, work=work)
    ref = ref_layer_norm_bwd(dh, x, mean, rstd, w, dsum)
    for name, got in (("dx", dx), ("dw", dw), ("db", db)):
        assert_within(got, *ref[name], name)
    assert untouched(dx)


@pytest.mark.parametrize("rows,cols", SIZES + [(5000, 1024), (2500, 513)])
@pytest.mark.parametrize("dt", TYPES)
def test_backward(rows, cols, dt):
    s, dh, dsum, w = make(rows, cols, dt, far=0.5), make(rows, cols, dt, seed=1), make(rows, cols, dt, seed=2), make(1, cols, dt, seed=3)[0]
    d = s.double() - s.double().mean(1, keepdim=True)
    mean, rstd = s.double().mean(1).float(), (d.square().mean(1) + 1e-5).rsqrt().float()
    work = torch.empty(sm.moe_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    for with_w, with_d in itertools.product((False, True), repeat=2):
        dx, dw, db = like(s), torch.empty_like(w), torch.empty_like(w)
        ww, dd = w if with_w else None, dsum if with_d else None
        sm.moe_layer_norm_bwd(dh, s, mean, rstd, dx=dx, w=ww, dsum=dd, dw=dw, db=db, work=work)
        ref = ref_layer_norm_bwd(dh, s, mean, rstd, ww, dd)
        for name, got in (("dx", dx), ("dw", dw), ("db", db)):
            assert_within(got, *ref[name], name)
    # parts of the results alone are the same
    for names in ({"dx"}, {"dw"}, {"db"}, {"dw", "db"}, {"dx", "db"}):
        out = {"dx": like(s), "dw": torch.empty_like(w), "db": torch.empty_like(w)}
        sm.moe_layer_norm_bwd(dh, s, mean, rstd, w=w, dsum=dsum, work=work, **{k: v for k, v in out.items() if k in names})
        for k in names:
            assert torch.equal(out[k], {"dx": dx, "dw": dw, "db": db}[k]), k


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("cols", [257, 4096, 20000])
def test_rows_far_from_zero(dt, cols):
    """A mean a thousand deviations away: the variance is not a difference of large numbers."""
    x = make(6, cols, torch.float32, far=1000.0).to(dt)
    h, rstd = like(x), torch.empty(6, device="cuda")
    sm.moe_layer_norm(x, h, rstd=rstd)
    ref = ref_layer_norm(x, None, None, None, 1e-5)
    assert_within(h, *ref["h"], "h")
    assert_within(rstd, *ref["rstd"], "rstd")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("cols", [64, 999, 4096, 9001])
def test_edges(dt, cols):
    x = make(6, cols, dt)
    x[1] = 3.0                 # constant: no deviation
    x[2, cols // 2] = float("inf")
    x[3, cols - 1] = float("nan")
    x[4] = 0.0
    h, mean, rstd = like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    sm.moe_layer_norm(x, h, mean=mean, rstd=rstd)
    assert bool((h[1] == 0).all()) and bool((h[4] == 0).all())
    assert float(mean[1]) == 3.0
    torch.testing.assert_close(rstd[1].double(), torch.tensor(1e-5 ** -0.5, device="cuda", dtype=torch.float64), rtol=1e-5, atol=0)
    assert bool(h[2].isnan().all()) and bool(h[3].isnan().all())
    ref = ref_layer_norm(x[[0, 5]], None, None, None, 1e-5)
    assert_within(h[[0, 5]], *ref["h"], "rows beside them")


@pytest.mark.parametrize("dt,size", [(torch.float32, 1e30), (torch.float32, 1e-30), (torch.bfloat16, 1e30), (torch.bfloat16, 1e-30),
                                     (torch.float16, 2e4), (torch.float16, 1e-6)])
@pytest.mark.parametrize("cols", [100, 1001, 4096, 9000, 40000])
def test_range(dt, size, cols):
    """Squares beyond the range of 32 bits; eps 0, so that the scale does not matter."""
    x = (make(4, cols, torch.float32) * size).to(dt)
    h, mean, rstd = like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    sm.moe_layer_norm(x, h, mean=mean, rstd=rstd, eps=0.0)
    inside = x.isfinite().all(1)  # (fp16: a few of them are beyond it)
    assert bool(h[~inside].isnan().all())
    ref = ref_layer_norm(x[inside], None, None, None, 0.0)
    for name, got in (("h", h), ("mean", mean), ("rstd", rstd)):
        assert_within(got[inside], *ref[name], name)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("cols", [72, 515, 4096, 8200])
def test_in_place(dt, cols):
    x, add, w = make(11, cols, dt), make(11, cols, dt, seed=1), make(1, cols, dt, seed=2)[0]
    h, total = like(x), like(x)
    mean, rstd = torch.empty(11, device="cuda"), torch.empty(11, device="cuda")
    sm.moe_layer_norm(x, h, w=w, add=add, sum=total, mean=mean, rstd=rstd)
    for into_h, into_sum in (("x", "add"), ("add", "x")):
        t = {"x": x.clone(), "add": add.clone()}
        sm.moe_layer_norm(t["x"], t[into_h], w=w, add=t["add"], sum=t[into_sum])
        assert torch.equal(t[into_h], h) and torch.equal(t[into_sum], total)
    dh, dsum = make(11, cols, dt, seed=3), make(11, cols, dt, seed=4)
    work = torch.empty(sm.moe_layer_norm_workspace(11, cols), dtype=torch.uint8, device="cuda")
    out = {"dx": like(x), "dw": torch.empty_like(w), "db": torch.empty_like(w)}
    sm.moe_layer_norm_bwd(dh, total, mean, rstd, w=w, dsum=dsum, work=work, **out)
    for into in ("dh", "s", "dsum"):
        t = {"dh": dh.clone(), "s": total.clone(), "dsum": dsum.clone()}
        dw, db = torch.empty_like(w), torch.empty_like(w)
        sm.moe_layer_norm_bwd(t["dh"], t["s"], mean, rstd, dx=t[into], w=w, dsum=t["dsum"], dw=dw, db=db, work=work)
        assert torch.equal(t[into], out["dx"]) and torch.equal(dw, out["dw"]) and torch.equal(db, out["db"]), into


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (2, 3), (7, 1), (8, 5)])
@pytest.mark.parametrize("cols", [1, 5, 33, 501, 1017, 4095, 8185, 8187])
def test_rows_alike_off_boundaries(cols, pad, shift, dt):
    """All tensors with the same rows' starts; NaN between the rows and in one of them reaches no other."""
    rows, bad = 60, 20
    good = [r for r in range(rows) if r != bad]

    def walled(t):
        out = torch.full((rows * (cols + pad) + shift,), float("nan"), device="cuda", dtype=dt)[shift:].as_strided((rows, cols), t.stride())
        return out.copy_(t)

    x, add, dh, dsum = (walled(make(rows, cols, dt, pad, shift, seed=i)) for i in range(4))
    w, b = make(1, cols, dt, 0, 1, seed=5)[0], make(1, cols, dt, 0, 0, seed=6)[0]
    h, total, dx = like(x), like(x), like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sm.moe_layer_norm(x, h, w=w, b=b, add=add, sum=total, mean=mean, rstd=rstd)
    ref = ref_layer_norm(x, w, b, add, 1e-5)
    for name, got in (("h", h), ("sum", total), ("mean", mean), ("rstd", rstd)):
        assert_within(got, *ref[name], name)
    assert untouched(h) and untouched(total)
    s = walled(total)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    work = torch.empty(sm.moe_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    sm.moe_layer_norm_bwd(dh, s, mean, rstd, dx=dx, w=w, dsum=dsum, dw=dw, db=db, work=work)
    ref = ref_layer_norm_bwd(dh, s, mean, rstd, w, dsum)
    for name, got in (("dx", dx), ("dw", dw), ("db", db)):
        assert_within(got, *ref[name], name)
    assert untouched(dx)

    clean = {"h": h[good], "sum": total[good], "dx": dx[good]}
    x[bad], dh[bad] = float("nan"), float("nan")
    sm.moe_layer_norm(x, h, w=w, b=b, add=add, sum=total)
    assert torch.equal(h[good], clean["h"]) and torch.equal(total[good], clean["sum"]) and bool(h[bad].isnan().all())
    sm.moe_layer_norm_bwd(dh, s, mean, rstd, dx=dh, w=w, dsum=dsum)  # over its own input
    assert torch.equal(dh[good], clean["dx"]) and bool(dh[bad].isnan().all())


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(40, 8193), (37, 16384), (50, 9001), (20, 20001), (18, 65536), (9, 65535), (5, 40000), (700, 8200)])
def test_gradient_of_long_rows(rows, cols, dt):
    """Rows that several blocks share, or that are walked again."""
    test_backward(rows, cols, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (7, 1)])
@pytest.mark.parametrize("cols", [8200, 16381, 33001])
def test_long_rows_alike_off_boundaries(cols, pad, shift, dt):
    test_rows_alike_off_boundaries(cols, pad, shift, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(12000, 129), (9001, 1033), (7000, 2051)])
def test_many_rows_off_boundaries(rows, cols, dt):
    """More rows than blocks: each block walks several."""
    test_forward(rows, cols, dt)
    test_backward(rows, cols, dt)


def test_gradient_against_differences():
    """In 32 bits: a step along a direction changes the loss by the gradient's share of it."""
    rows, cols = 5, 192
    x, add = make(rows, cols, torch.float32), make(rows, cols, torch.float32, seed=1)
    w, b, g = make(1, cols, torch.float32, seed=2)[0], make(1, cols, torch.float32, seed=3)[0], make(rows, cols, torch.float32, seed=4)
    h, total = like(x), like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    sm.moe_layer_norm(x, h, w=w, b=b, add=add, sum=total, mean=mean, rstd=rstd)
    dx, dw, db = like(x), torch.empty_like(w), torch.empty_like(b)
    work = torch.empty(sm.moe_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    sm.moe_layer_norm_bwd(g, total, mean, rstd, dx=dx, w=w, dw=dw, db=db, work=work)

    def loss(x, w, b):
        s = x.double() + add.double()
        n = (s - s.mean(1, keepdim=True)) / (s.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
        return ((n * w.double() + b.double()) * g.double()).sum()

    for i, (name, grad) in enumerate((("x", dx), ("w", dw), ("b", db))):
        at = {"x": x, "w": w, "b": b}
        step = torch.randn(at[name].shape, generator=torch.Generator("cuda").manual_seed(9 + i), device="cuda").double() * 1e-4
        ends = [loss(**dict(at, **{name: at[name].double() + k * step})) for k in (1, -1)]
        diff = float(ends[0] - ends[1]) / 2
        share = float((grad.double() * step).sum())
        # third-order remainder of a step of 1e-4 a column, and the gradient's own roundings
        assert abs(diff - share) <= 1e-6 * float((grad.double() * step).abs().sum()) + 1e-8, name


def test_repeats_and_captures():
    x, w = make(3000, 1024, torch.bfloat16), make(1, 1024, torch.bfloat16, seed=1)[0]
    dh = make(3000, 1024, torch.bfloat16, seed=2)
    h, mean, rstd = like(x), torch.empty(3000, device="cuda"), torch.empty(3000, device="cuda")
    dx, dw, db = like(x), torch.empty_like(w), torch.empty_like(w)
    work = torch.empty(sm.moe_layer_norm_workspace(3000, 1024), dtype=torch.uint8, device="cuda")

    def both():
        sm.moe_layer_norm(x, h, w=w, mean=mean, rstd=rstd)
        sm.moe_layer_norm_bwd(dh, x, mean, rstd, dx=dx, w=w, dw=dw, db=db, work=work)

    both()
    first = [t.clone() for t in (h, dx, dw, db)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
        with torch.cuda.graph(graph, stream=side):
            both()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in (h, dx, dw, db):
            t.zero_()
        work.fill_(255)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, (h, dx, dw, db)))


def test_no_rows():
    e, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    none = torch.empty(0, device="cuda")
    dw, db = torch.full((64,), 5.0, device="cuda"), torch.full((64,), 5.0, device="cuda")
    sm.moe_layer_norm(e, e, w=w)
    sm.moe_layer_norm_bwd(e, e, none, none, dx=e, w=w, dw=dw, db=db)
    assert not dw.any() and not db.any()


def test_parts_of_the_forward():
    """Every output may be left out; what is there is the same."""
    x, add, w = make(5, 1000, torch.bfloat16), make(5, 1000, torch.bfloat16, seed=1), make(1, 1000, torch.bfloat16, seed=2)[0]
    full = {"h": like(x), "sum": like(x), "mean": torch.empty(5, device="cuda"), "rstd": torch.empty(5, device="cuda")}
    sm.moe_layer_norm(x, w=w, add=add, **full)
    for name in full:
        one = torch.empty_like(full[name])
        sm.moe_layer_norm(x, w=w, add=add, **{name: one})
        assert torch.equal(one, full[name]), name


def test_refusals():
    x, w = make(4, 64, torch.bfloat16), make(1, 64, torch.bfloat16)[0]
    h, st = like(x), torch.empty(4, device="cuda")
    work = torch.empty(sm.moe_layer_norm_workspace(4, 64), dtype=torch.uint8, device="cuda")
    bad = [lambda: sm.moe_layer_norm(x), lambda: sm.moe_layer_norm(x, h[:3]), lambda: sm.moe_layer_norm(x, h.float()),
           lambda: sm.moe_layer_norm(x, h, w=w[:63]), lambda: sm.moe_layer_norm(x, h, w=w.float()), lambda: sm.moe_layer_norm(x, h, mean=st[:3]),
           lambda: sm.moe_layer_norm(x, h, sum=h), lambda: sm.moe_layer_norm(x.cpu(), h), lambda: sm.moe_layer_norm(x, h.cpu()),
           lambda: sm.moe_layer_norm(x[0], h[0]), lambda: sm.moe_layer_norm(x.t(), h.t()), lambda: sm.moe_layer_norm(x, h, eps=-1.0),
           lambda: sm.moe_layer_norm(x.double(), h.double()), lambda: sm.moe_layer_norm(x[:1].expand(4, 64), h),
           lambda: sm.moe_layer_norm_bwd(x, x, st, st), lambda: sm.moe_layer_norm_bwd(x, x, None, st, dx=h),
           lambda: sm.moe_layer_norm_bwd(x, None, st, st, dx=h), lambda: sm.moe_layer_norm_bwd(x, x, st, st[:2], dx=h),
           lambda: sm.moe_layer_norm_bwd(x, x, st, st, dw=w, work=work.cpu())]
    for i, call in enumerate(bad):
        with pytest.raises(sm.SymmoeError) as e:
            call()
        assert e.value.code == sm.SYM_EINVAL, i
    for short in (None, work[:work.numel() - 16]):
        with pytest.raises(sm.SymmoeError) as e:
            sm.moe_layer_norm_bwd(x, x, st, st, dw=torch.empty_like(w), work=short)
        assert e.value.code == sm.SYM_ENOSPACE
    sm.moe_layer_norm_bwd(x, x, st, st, dx=h)  # dx alone wants no workspace
