"""What dropout drops between a block without a norm and the stream passes
nothing on, whatever it holds: the same bits come out, forward and backward, as
with zeros in its place, in every norm kernel."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import kept

pytestmark = pytest.mark.gpu

COLS = [256, 4096, 5120, 7168, 333, 4095, 9000, 9001]
P, SEED, OFFSET = 0.4, 21, 22


def call(o, x, dy, dh, gate, w_pre, act):
    (rows, cols), like = o.shape, torch.empty_like
    kw = dict(o=o, gate=gate, gate_act=act if gate is not None else "none", scale=0.7, p=P, seed=SEED, offset=OFFSET,
              post_norm=False, w_pre=w_pre)
    out = dict(y=like(x), h=like(x), rstd_pre=torch.empty(rows, device="cuda"))
    sm.moe_block_norm(x, **out, **kw)
    grads = dict(dx=like(x), do=like(x), dw_pre=like(w_pre), dgate=None if gate is None else like(gate))
    G = 0 if gate is None else len(gate)
    work = torch.empty(sm.moe_block_norm_workspace(rows, cols, G), dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=dy, dh=dh, y=out["y"], rstd_pre=out["rstd_pre"], work=work, **grads, **kw)
    return {**out, **grads}


@pytest.mark.parametrize("gates", [0, 1, 6])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_dropped_garbage_passes_nothing_on(cols, dt, gates):
    gen = torch.Generator(device="cuda").manual_seed(cols + gates)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    rows = 6
    o, x, dy, dh = (randn(rows, cols) for _ in range(4))
    gate, w_pre = randn(gates, cols) if gates else None, (1 + 0.2 * randn(cols)).to(dt)
    keep = kept(SEED, OFFSET, o.shape, P)
    clean = call(torch.where(keep, o, torch.zeros_like(o)), x, dy, dh, gate, w_pre, "sigmoid")
    garbage = torch.where(o > 0.5, float("inf"), torch.where(o < -0.5, -float("inf"), float("nan"))).to(dt)
    dirty = call(torch.where(keep, o, garbage), x, dy, dh, gate, w_pre, "sigmoid")
    for name, t in clean.items():
        if t is not None:
            assert bool(t.isfinite().all()) and torch.equal(t, dirty[name]), name


@pytest.mark.parametrize("gates", [0, 1, 6])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_a_dropped_infinity_before_the_norm(cols, dt, gates):
    """The norm after the block makes zeros of the row with the infinity; the other
    rows, and what is summed over rows, do not see it."""
    gen = torch.Generator(device="cuda").manual_seed(cols + gates)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    rows, row = 6, 2
    o, x, dy = (randn(rows, cols) for _ in range(3))
    gate, like = randn(gates, cols) if gates else None, torch.empty_like
    at = int((~kept(SEED, OFFSET, o.shape, P))[row].nonzero()[-1])
    got = []
    for dirty in (True, False):
        o[row] = randn(cols) if dirty else 0
        if dirty:
            o[row, at] = -float("inf")
        kw = dict(o=o, gate=gate, gate_act="tanh" if gates else "none", scale=0.7, p=P, seed=SEED, offset=OFFSET)
        y, h, ro = like(x), like(x), torch.empty(rows, device="cuda")
        sm.moe_block_norm(x, y=y, h=h, rstd_post=ro, **kw)
        assert dirty == (float(ro[row]) == 0)
        ro[row] = 0
        grads = dict(dx=like(x), do=like(x), dw_post=torch.empty(cols, device="cuda", dtype=dt),
                     dgate=None if gate is None else like(gate))
        work = torch.empty(sm.moe_block_norm_workspace(rows, cols, gates), dtype=torch.uint8, device="cuda")
        sm.moe_block_norm_bwd(dy=dy, rstd_post=ro, work=work, **grads, **kw)
        got.append(dict(y=y, h=h, rstd_post=ro, **grads))
    assert torch.equal(got[0]["y"][row], x[row]) and bool((got[0]["do"][row] == 0).all())
    for name, t in got[1].items():
        if t is not None:
            assert bool(t.isfinite().all()) and torch.equal(t, got[0][name]), name


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_without_a_norm_the_gradient_does_not_depend_on_the_block_output(cols, dt):
    """y = x + scale * o: do = scale * dy, at an infinite o too."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    dy = torch.randn(3, cols, generator=gen, device="cuda").to(dt)
    o = torch.full_like(dy, float("inf"))
    do, work = torch.empty_like(dy), torch.empty(sm.moe_block_norm_workspace(3, cols), dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=dy, o=o, do=do, scale=0.5, post_norm=False, work=work)
    assert torch.equal(do, 0.5 * dy)
