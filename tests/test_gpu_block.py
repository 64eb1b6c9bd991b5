"""SwiGLU of expert rows, counter-based dropout and the norms around a block
against their definitions in 64 bits, their gradients also against
differences of those definitions."""
import itertools

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import (EVAL, assert_within, kept, ref_norm, ref_norm_bwd, ref_swiglu, ref_swiglu_bwd)

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(gen, shape, dtype, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def laid(t, how):
    """The tensor as it is, in rows 16-byte aligned but padded, or off every boundary."""
    if how == "plain":
        return t.contiguous()
    pad = 16 if how == "padded" else 3
    room = torch.full((*t.shape[:-1], (t.shape[-1] + 7) // 8 * 8 + pad), NAN, device="cuda", dtype=t.dtype)
    v = room[..., :t.shape[-1]] if how == "padded" else room[..., 1:1 + t.shape[-1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ swiglu
SHAPES = [(1, 1, 1), (1, 1, 128), (1, 37, 2048), (2, 5, 333), (1, 130, 4104), (3, 9, 24), (1, 2, 65536)]


@pytest.mark.parametrize("how", ["plain", "padded", "odd"])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", SHAPES)
def test_swiglu(shape, dt, how):
    gen = gen_of(sum(shape))
    g, u, dh = (laid(randn(gen, shape, dt, 1.5), how) for _ in range(3))
    w = torch.rand(shape[:2], generator=gen, device="cuda")
    h = laid(torch.zeros(shape, device="cuda", dtype=dt), how)
    sm.moe_swiglu_rows(g, u, h, row_w=w)
    ref = ref_swiglu(g, u, w)
    assert_within(h, ref, ref.abs(), "h")
    dg, du = (laid(torch.zeros(shape, device="cuda", dtype=dt), how) for _ in range(2))
    dw = torch.full(shape[:2], NAN, device="cuda")
    sm.moe_swiglu_rows_bwd(g, u, dh, dg, du, row_w=w, d_row_w=dw)
    for got, (ref, mag), name in zip((dg, du, dw), ref_swiglu_bwd(g, u, dh, w), ("dg", "du", "d_row_w")):
        assert_within(got, ref, mag, name)
    # without weights, in place
    ref, mag = ref_swiglu_bwd(g, u, dh, torch.ones_like(w))[0]
    sm.moe_swiglu_rows_bwd(g, u, dh, g, du)
    assert_within(g, ref, mag, "dg in place")


def test_swiglu_mixed_layouts_and_totals():
    """Tensors whose rows start at different places of a line; rows past a slot's total stay."""
    gen = gen_of(1)
    shape = (3, 40, 200)
    g, u = laid(randn(gen, shape, BF16), "plain"), laid(randn(gen, shape, BF16), "odd")
    h = torch.full(shape, 7.0, device="cuda", dtype=BF16)
    total = torch.tensor([0, 13, 99], dtype=torch.int32, device="cuda")  # 99: cut to 40
    sm.moe_swiglu_rows(g, u, h, total=total)
    ref = ref_swiglu(g, u, torch.ones(shape[:2], device="cuda"))
    for d, n in enumerate((0, 13, 40)):
        assert bool((h[d, n:] == 7.0).all())
        assert_within(h[d, :n], ref[d, :n], ref[d, :n].abs(), "h")
    total[1] = -5
    h.fill_(7.0)
    sm.moe_swiglu_rows(g, u, h, total=total)
    assert bool((h[1] == 7.0).all())


def test_swiglu_far_from_zero():
    """exp overflows and underflows on the way: the limits come out."""
    g = torch.tensor([[-1e4, -200.0, -90.0, 90.0, 200.0, 1e4]], device="cuda")
    u = torch.full_like(g, 2.0)
    h, dg, du = (torch.empty_like(g) for _ in range(3))
    sm.moe_swiglu_rows(g, u, h)
    sm.moe_swiglu_rows_bwd(g, u, torch.ones_like(g), dg, du)
    assert h.tolist()[0][3:] == [180.0, 400.0, 2e4] and float(h[0, :3].abs().max()) < 1e-30
    assert dg.tolist()[0][3:] == [2.0, 2.0, 2.0] and float(dg[0, :3].abs().max()) < 1e-30
    assert du.tolist()[0][3:] == [90.0, 200.0, 1e4]


def test_swiglu_gradient_against_differences():
    gen = gen_of(2)
    shape = (1, 6, 96)
    g, u, dh = (randn(gen, shape, FP32) for _ in range(3))
    w = torch.rand(shape[:2], generator=gen, device="cuda")
    dg, du, dw = torch.empty_like(g), torch.empty_like(u), torch.empty_like(w)
    sm.moe_swiglu_rows_bwd(g, u, dh, dg, du, row_w=w, d_row_w=dw)
    directional(lambda a, b, c: (ref_swiglu(a, b, c) * dh.double()).sum(), (g, u, w), (dg, du, dw), gen)


def directional(loss, inputs, grads, gen):
    """(loss(x + h v) - loss(x - h v)) / 2h along random directions, in 64 bits
    (error h^2 times third derivatives of order one per element, plus 1e-16 /
    h), against the inner product of v with the computed gradient (error at
    most EVAL of the sizes' product)."""
    inputs = [t.double() for t in inputs]
    h = 1e-5
    for _ in range(4):
        vs = [torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for t in inputs]
        up = loss(*(t + h * v for t, v in zip(inputs, vs)))
        down = loss(*(t - h * v for t, v in zip(inputs, vs)))
        want = float((up - down) / (2 * h))
        got = sum(float((v * g.double()).sum()) for v, g in zip(vs, grads))
        size = sum(float((v * g.double()).abs().sum()) for v, g in zip(vs, grads))
        assert abs(got - want) <= 10 * EVAL * size + 1e-6, (got, want, size)


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("how", ["plain", "padded", "odd"])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7168), (33, 1001), (17, 130), (1000, 8), (3, 65536)])
def test_dropout(shape, dt, how):
    gen = gen_of(sum(shape))
    x, res = (laid(randn(gen, shape, dt), how) for _ in range(2))
    seed, offset, p = 0x1234_5678_9ABC_DEF0, (1 << 40) + 5, 0.3
    y = laid(torch.zeros(shape, device="cuda", dtype=dt), how)
    keep = kept(seed, offset, shape, p)
    ref = torch.where(keep, x.double() / (1 - p), 0.0)
    sm.moe_dropout(x, y, p, seed, offset)
    assert_within(y, ref, ref.abs(), "dropout")
    assert torch.equal(y == 0, ~keep | (x == 0))
    sm.moe_dropout(x, y, p, seed, offset, residual=res)
    assert_within(y, ref + res.double(), ref.abs() + res.double().abs(), "dropout + residual")
    again = y.clone()
    sm.moe_dropout(x, x, p, seed, offset, residual=res)  # in place
    assert torch.equal(x, again)


def test_dropout_known_words():
    """The generator's published first block: zero key, zero counter."""
    words = [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    x, y = torch.ones(1, 4, device="cuda"), torch.empty(1, 4, device="cuda")
    for i, w in enumerate(words):
        sm.moe_dropout(x, y, w / 2 ** 32, 0, 0)          # kept at the word itself ...
        assert float(y[0, i]) != 0
        sm.moe_dropout(x, y, (w + 1) / 2 ** 32, 0, 0)    # ... dropped one above it
        assert float(y[0, i]) == 0


def test_dropout_zero_probability_and_masked_garbage():
    gen = gen_of(4)
    x = randn(gen, (9, 257), FP32)
    y = torch.empty_like(x)
    sm.moe_dropout(x, y, 0.0, 1)
    assert torch.equal(x, y)
    keep = kept(1, 2, x.shape, 0.5)
    dirty = torch.where(keep, x, torch.where(x > 0, float("inf"), NAN))
    sm.moe_dropout(dirty, y, 0.5, 1, 2)
    assert bool(y.isfinite().all()) and bool((y[~keep] == 0).all())


def test_dropout_slots_and_long_tensors():
    """Element indices run over the slots, and past 2^32."""
    gen = gen_of(6)
    x = randn(gen, (3, 5, 12), FP32)
    y, flat = torch.empty_like(x), torch.empty(15, 12, device="cuda")
    sm.moe_dropout(x, y, 0.5, 3)
    sm.moe_dropout(x.view(15, 12), flat, 0.5, 3)
    assert torch.equal(y.view(15, 12), flat)
    rows, cols = 65540, 65536
    big = torch.ones(rows, cols, device="cuda", dtype=BF16)
    sm.moe_dropout(big, big, 0.5, 9)
    # the last rows: blocks from (rows - 2) * cols / 4 on, whose counter's
    # second word is not zero
    import numpy as np
    first = (rows - 2) * cols // 4
    i = np.arange(first, first + cols // 2, dtype=np.uint64)
    m, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    c, k = [i & m, i >> s32, np.zeros_like(i), np.zeros_like(i)], [9, 0]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & m, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    want = torch.from_numpy(np.stack(c, 1).reshape(2, cols) >= np.uint64(1 << 31)).cuda()
    assert torch.equal(big[-2:] != 0, want)


# ------------------------------------------------------------------ norms
NORMS = [
    # rows, cols, gate rows (0: none), activation, dropout, post weight, pre weight, post norm, block output, next norm
    (1, 7168, 1, "none", 0.0, True, True, True, True, True),
    (5, 128, 5, "sigmoid", 0.1, True, True, True, True, True),
    (12, 1000, 3, "tanh", 0.25, True, False, True, True, True),
    (700, 256, 2, "sigmoid", 0.1, False, True, True, True, True),
    (9, 2056, 0, "none", 0.1, True, True, True, True, False),
    (7, 520, 1, "tanh", 0.0, False, True, False, True, True),
    (33, 4096, 0, "none", 0.0, False, True, True, False, True),
    (3, 20480, 1, "tanh", 0.1, True, True, True, True, True),
    (2, 65536, 2, "sigmoid", 0.0, True, True, True, True, True),
    (40, 333, 4, "sigmoid", 0.2, True, True, True, True, True),
    (6, 1, 1, "tanh", 0.0, True, True, True, True, True),
    (3, 9001, 1, "none", 0.1, True, True, True, True, True),
    (4, 5001, 2, "tanh", 0.1, True, True, True, True, True),
    (350, 1023, 7, "sigmoid", 0.1, True, True, True, True, True),
    (1200, 512, 300, "tanh", 0.1, True, True, True, True, True),
    (900, 264, 900, "sigmoid", 0.0, True, True, True, True, True),
    (310, 8192, 5, "tanh", 0.1, True, True, True, True, True),
    # many rows a block, of changing alignment
    (1300, 4095, 1, "tanh", 0.1, True, True, True, True, True),
    (640, 8191, 2, "sigmoid", 0.1, True, True, True, True, True),
    (700, 6001, 700, "tanh", 0.2, True, False, True, True, True),
    (3000, 1001, 750, "none", 0.1, True, True, True, True, True),
    (20000, 31, 4, "sigmoid", 0.5, False, True, True, True, True),
    (500, 7167, 0, "none", 0.0, True, True, True, False, True),
    (810, 2047, 0, "none", 0.1, True, True, False, True, False),
]


def norm_case(i, dt, how):
    rows, cols, G, act, p, has_wo, has_wp, post, has_o, has_h = NORMS[i]
    gen = gen_of(50 + i)
    one = lambda: laid(randn(gen, (rows, cols), dt), how)  # noqa: E731
    vec = lambda: randn(gen, (cols,), dt, 0.3).add_(1)  # noqa: E731
    kw = dict(o=one() if has_o else None, w_post=vec() if has_o and post and has_wo else None,
              gate=laid(randn(gen, (G, cols), dt), how) if has_o and G else None, gate_act=act if G else "none",
              scale=0.6, p=p, seed=77 + i, offset=i, w_pre=vec() if has_h and has_wp else None, post_norm=post)
    return gen, one, rows, cols, kw, post and has_o, has_o, has_h


@pytest.mark.parametrize("how", ["plain", "padded", "odd"])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("i", range(len(NORMS)))
def test_block_norm(i, dt, how):
    gen, one, rows, cols, kw, post, has_o, has_h = norm_case(i, dt, how)
    x = one()
    room = lambda: laid(torch.zeros(rows, cols, device="cuda", dtype=dt), how)  # noqa: E731
    stat = lambda want: torch.full((rows,), NAN, device="cuda") if want else None  # noqa: E731
    y, h = room() if has_o else None, room() if has_h else None
    ro, ry = stat(post), stat(has_h)
    sm.moe_block_norm(x, y=y, h=h, rstd_post=ro, rstd_pre=ry, **kw)
    ref, mag = ref_norm(x, **kw)
    if has_o:
        assert_within(y, ref["y"], mag["y"], "y")
    if has_h:
        assert_within(h, ref["h"], mag["h"] + ref["h"].abs(), "h")
        assert_within(ry, ref["rstd_pre"], ref["rstd_pre"], "rstd_pre")
    if post:
        assert_within(ro, ref["rstd_post"], ref["rstd_post"], "rstd_post")
    if has_o:  # in place
        first = y.clone()
        sm.moe_block_norm(x, y=x, h=h, **kw)
        assert torch.equal(x, first)


@pytest.mark.parametrize("how", ["plain", "padded", "odd"])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
@pytest.mark.parametrize("i", range(len(NORMS)))
def test_block_norm_gradient(i, dt, how):
    gen, one, rows, cols, kw, post, has_o, has_h = norm_case(i, dt, how)
    y, dy, dh = one(), one(), one() if has_h else None
    ro = (kw["o"].double().square().mean(1) + 1e-6).rsqrt().float() if post else None
    ry = (y.double().square().mean(1) + 1e-6).rsqrt().float() if has_h else None
    kw.update(rstd_post=ro, rstd_pre=ry)
    G = 0 if kw["gate"] is None else kw["gate"].shape[0]
    room = lambda: laid(torch.zeros(rows, cols, device="cuda", dtype=dt), how)  # noqa: E731
    vec = lambda: torch.full((cols,), NAN, device="cuda", dtype=dt)  # noqa: E731
    got = dict(dx=room(), do=room() if has_o else None, dw_pre=vec() if has_h else None, dw_post=vec() if post else None,
               dgate=laid(torch.zeros(G, cols, device="cuda", dtype=dt), how) if G else None)
    work = torch.full((sm.moe_block_norm_workspace(rows, cols, G),), 0xFF, dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=dy, dh=dh, y=y if has_h else None, work=work, **got, **kw)
    ref = ref_norm_bwd(dy, dh, y, **{k: v for k, v in kw.items()})
    for name, t in got.items():
        if t is not None:
            assert_within(t, *ref[name], name)
    # the same bits again, also with dx in place of dy
    twice = {k: None if v is None else torch.empty_like(v) for k, v in got.items()}
    twice["dx"] = dy
    sm.moe_block_norm_bwd(dy=dy, dh=dh, y=y if has_h else None, work=work, **twice, **kw)
    for name, t in got.items():
        assert t is None or torch.equal(t, twice[name]), name


@pytest.mark.parametrize("act,p,G", list(itertools.product(["none", "sigmoid", "tanh"], [0.0, 0.2], [1, 4])))
def test_block_norm_gradient_against_differences(act, p, G):
    gen = gen_of(8)
    R, C = 8, 64
    x, o, dy, dh = (randn(gen, (R, C), FP32) for _ in range(4))
    wo, wp = (randn(gen, (C,), FP32, 0.3) + 1 for _ in range(2))
    gate = randn(gen, (G, C), FP32)
    kw = dict(gate_act=act, scale=0.8, p=p, seed=5, offset=6)
    y, h = torch.empty_like(x), torch.empty_like(x)
    ro, ry = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    sm.moe_block_norm(x, o=o, w_post=wo, gate=gate, y=y, w_pre=wp, h=h, rstd_post=ro, rstd_pre=ry, **kw)
    dx, do, dwp, dwo, dg = (torch.empty_like(t) for t in (x, o, wp, wo, gate))
    work = torch.empty(sm.moe_block_norm_workspace(R, C, G), dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=dy, dh=dh, y=y, o=o, w_post=wo, gate=gate, w_pre=wp, rstd_post=ro, rstd_pre=ry,
                          dx=dx, do=do, dw_pre=dwp, dw_post=dwo, dgate=dg, work=work, **kw)

    def loss(x, o, wp, wo, gate):
        ref, _ = ref_norm(x, o, wo, gate, w_pre=wp, **kw)
        return (ref["y"] * dy.double()).sum() + (ref["h"] * dh.double()).sum()

    directional(loss, (x, o, wp, wo, gate), (dx, do, dwp, dwo, dg), gen)


def test_block_norm_where_the_block_cancels_the_stream():
    """x + scale * norm(o) nearly 0: y's norm is far below its parts' (the sum of
    y^2 may not come from their sums)."""
    gen = gen_of(12)
    for rows, cols in ((5, 1024), (3, 4096), (4, 333), (2, 10000)):
        o = randn(gen, (rows, cols), FP32)
        n = o.double() * (o.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
        x = (-0.5 * n + 1e-3 * torch.randn(n.shape, generator=gen, device="cuda", dtype=torch.float64)).float()
        y, h, ry = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
        sm.moe_block_norm(x, o=o, y=y, h=h, scale=0.5, rstd_pre=ry)
        ref, mag = ref_norm(x, o=o, scale=0.5)
        assert_within(y, ref["y"], mag["y"], "y")
        # y itself is off by EVAL of its parts (about 0.5), 500 times its size;
        # its norm by that much less the square root of the row's length
        assert float((ry.double() / ref["rstd_pre"] - 1).abs().max()) < 500 * EVAL / 10


def test_block_norm_rows_of_zeros_and_parts():
    x = torch.zeros(4, 256, device="cuda")
    h, ry = torch.full_like(x, NAN), torch.empty(4, device="cuda")
    sm.moe_block_norm(x, h=h, rstd_pre=ry)
    assert bool((h == 0).all()) and torch.allclose(ry, torch.full_like(ry, 1e3))
    # a gradient without the stream's part, and one without the next norm's
    gen = gen_of(10)
    y, d = randn(gen, (4, 256), FP32), randn(gen, (4, 256), FP32)
    ry = (y.double().square().mean(1) + 1e-6).rsqrt().float()
    work = torch.empty(sm.moe_block_norm_workspace(4, 256), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(y)
    none = dict(o=None, w_post=None, gate=None, gate_act="none", scale=1.0, p=0.0, seed=0, offset=0, w_pre=None)
    sm.moe_block_norm_bwd(dh=d, y=y, rstd_pre=ry, dx=dx, work=work)
    assert_within(dx, *ref_norm_bwd(None, d, y, rstd_post=None, rstd_pre=ry, **none)["dx"], "dx")
    do = torch.empty_like(y)
    sm.moe_block_norm_bwd(dy=d, o=y, rstd_post=ry, dx=dx, do=do, work=work)
    assert torch.equal(dx, d)
    assert_within(do, *ref_norm_bwd(d, None, None, **dict(none, o=y), rstd_post=ry, rstd_pre=None)["do"], "do")


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    sm.moe_block_norm(x, h=x)
    sm.moe_dropout(x, x, 0.5, 1)
    sm.moe_swiglu_rows(x, x, x)
    dw, dg = torch.full((64,), NAN, device="cuda"), torch.full((2, 64), NAN, device="cuda")
    e = torch.empty(0, device="cuda")
    sm.moe_block_norm_bwd(dy=x, dh=x, y=x, o=x, gate=dg.clone(), rstd_post=e, rstd_pre=e, dx=x, do=x, dw_pre=dw, dgate=dg)
    assert bool((dw == 0).all()) and bool((dg == 0).all())


def _raises(code, call, *a, **kw):
    with pytest.raises(sm.SymmoeError) as ei:
        call(*a, **kw)
    assert ei.value.code == code


def test_refusals():
    x, b = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda", dtype=BF16)
    v = torch.zeros(4, device="cuda")
    EINVAL = sm.SYM_EINVAL
    _raises(EINVAL, sm.moe_dropout, x, x, 1.0, 0)
    _raises(EINVAL, sm.moe_dropout, x, x, -0.1, 0)
    _raises(EINVAL, sm.moe_dropout, x, x, NAN, 0)
    _raises(EINVAL, sm.moe_dropout, x, b, 0.1, 0)
    _raises(EINVAL, sm.moe_dropout, x.double(), x.double(), 0.1, 0)
    _raises(EINVAL, sm.moe_dropout, x.cpu(), x.cpu(), 0.1, 0)
    _raises(EINVAL, sm.moe_dropout, x.T, x.T, 0.1, 0)
    _raises(EINVAL, sm.moe_dropout, x, x[:, :32], 0.1, 0)
    _raises(EINVAL, sm.moe_swiglu_rows, x, b, x)
    _raises(EINVAL, sm.moe_swiglu_rows, x, x, x[:2])
    _raises(EINVAL, sm.moe_swiglu_rows, x, x, x, row_w=v[:3])
    _raises(EINVAL, sm.moe_swiglu_rows, x, x, x, row_w=v.double())
    _raises(EINVAL, sm.moe_swiglu_rows, x, x, x, total=torch.zeros(2, dtype=torch.int32, device="cuda"))
    _raises(EINVAL, sm.moe_swiglu_rows_bwd, x, x, x, x, b)
    _raises(EINVAL, sm.moe_block_norm, x)                                     # nothing to write
    _raises(EINVAL, sm.moe_block_norm, x, o=x, h=x)                           # a block output, but no stream after it
    _raises(EINVAL, sm.moe_block_norm, x, y=x, h=x)                           # a stream after no block
    _raises(EINVAL, sm.moe_block_norm, x, o=x, y=x, gate=x[:3])               # 3 does not divide 4
    _raises(EINVAL, sm.moe_block_norm, x, o=x, y=x, gate=x[:1], gate_act="relu")
    _raises(EINVAL, sm.moe_block_norm, x, o=x, y=x, p=1.0)
    _raises(EINVAL, sm.moe_block_norm, x, h=x, eps=-1.0)
    _raises(EINVAL, sm.moe_block_norm, x, o=b, y=x)
    _raises(EINVAL, sm.moe_block_norm, x, o=x, y=x, post_norm=False, w_post=x[0])
    _raises(EINVAL, sm.moe_block_norm, x, h=x, w_pre=x[0, :32])
    work = torch.zeros(sm.moe_block_norm_workspace(4, 64, 1), dtype=torch.uint8, device="cuda")
    _raises(EINVAL, sm.moe_block_norm_bwd, dx=x, work=work)                   # no gradient comes in
    _raises(EINVAL, sm.moe_block_norm_bwd, dh=x, dx=x, work=work)             # y, rstd_pre missing
    _raises(EINVAL, sm.moe_block_norm_bwd, dy=x, o=x, do=x, work=work)        # rstd_post missing
    _raises(EINVAL, sm.moe_block_norm_bwd, dy=x, o=x, rstd_post=v, dgate=x[:1], work=work)
    _raises(sm.SYM_ENOSPACE, sm.moe_block_norm_bwd, dy=x, o=x, rstd_post=v, do=x)
    _raises(sm.SYM_ENOSPACE, sm.moe_block_norm_bwd, dy=x, o=x, rstd_post=v, do=x, work=work[:16])
