"""Block norms of values near the ends of a type's range: what is normalised or
gated on the way has to stay in range wherever the definition's own steps do."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import assert_within, ref_norm, ref_norm_bwd

pytestmark = pytest.mark.gpu

COLS = [256, 4096, 5120, 7168, 333, 4095, 9000, 9001]
ROWS = 7
# name: (size of o, size of the gate or 0 for none, size of x, eps)
FORWARD = {
    "gated squares above the range": (1e15, 1e7, 1e6, 1e-6),
    "gated squares below the range": (1e-13, 1e-12, 0.0, 0.0),
    "gated squares below the range, beside a stream": (1e-13, 1e-12, 1e-13, 0.0),
    "gated products above the range": (1e16, 1e16, 1e15, 1e-6),
    "large rows": (1e16, 0, 1.0, 1e-6),
    "small rows": (1e-16, 0, 1.0, 0.0),
}


def inputs(cols, dt, o_size, gate_size, x_size):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    o, x = (o_size * randn(ROWS, cols)).to(dt), (x_size * randn(ROWS, cols)).to(dt)
    gate = (gate_size * (1 + 0.3 * randn(1, cols))).to(dt) if gate_size else None
    return gen, o, x, gate, (1 + 0.2 * randn(cols)).to(dt), (1 + 0.2 * randn(cols)).to(dt)


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", FORWARD)
def test_forward(name, cols, dt, p):
    o_size, gate_size, x_size, eps = FORWARD[name]
    _, o, x, gate, w_post, w_pre = inputs(cols, dt, o_size, gate_size, x_size)
    kw = dict(o=o, gate=gate, w_post=w_post, w_pre=w_pre, scale=0.7, p=p, seed=1, offset=2, eps=eps)
    out = dict(y=torch.empty_like(x), h=torch.empty_like(x), rstd_post=torch.empty(ROWS, device="cuda"),
               rstd_pre=torch.empty(ROWS, device="cuda"))
    sm.moe_block_norm(x, **out, **kw)
    ref, mag = ref_norm(x, **kw)
    assert_within(out["y"], ref["y"], mag["y"], "y")
    assert_within(out["h"], ref["h"], mag["h"] + ref["h"].abs(), "h")
    assert_within(out["rstd_post"], ref["rstd_post"], ref["rstd_post"], "rstd_post")
    assert_within(out["rstd_pre"], ref["rstd_pre"], ref["rstd_pre"], "rstd_pre")


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_products_beyond_the_range_before_the_norm(cols, dt, p):
    """o times the gate is above the type's range, their normalised product is not."""
    _, o, x, gate, w_post, _ = inputs(cols, dt, 1e17, 1e23, 1e22)
    kw = dict(o=o, gate=gate, w_post=w_post, scale=0.7, p=p, seed=1, offset=2)
    y = torch.empty_like(x)
    sm.moe_block_norm(x, y=y, **kw)
    ref, mag = ref_norm(x, **kw)
    assert_within(y, ref["y"], mag["y"], "y")


# name: (size of o, size of the gate or 0 for none)
BACKWARD = {"small rows": (1e-14, 0), "large rows": (1e15, 0), "large rows, large gate": (1e17, 1e20),
            "small rows, small gate": (1e-14, 1e-10)}


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("name", BACKWARD)
def test_backward(name, cols, dt, p):
    o_size, gate_size = BACKWARD[name]
    gen, o, _, gate, w_post, w_pre = inputs(cols, dt, o_size, gate_size, 1.0)
    y, dy, dh = (torch.randn(ROWS, cols, generator=gen, device="cuda").to(dt) for _ in range(3))
    kw = dict(o=o, gate=gate, gate_act="none", w_post=w_post, w_pre=w_pre, scale=0.7, p=p, seed=1, offset=2,
              rstd_post=o.double().square().mean(1).rsqrt().float(), rstd_pre=y.double().square().mean(1).rsqrt().float())
    like = torch.empty_like
    got = dict(dx=like(y), do=like(o), dw_pre=like(w_pre), dw_post=like(w_post), dgate=None if gate is None else like(gate))
    work = torch.empty(sm.moe_block_norm_workspace(ROWS, cols, 0 if gate is None else 1), dtype=torch.uint8, device="cuda")
    sm.moe_block_norm_bwd(dy=dy, dh=dh, y=y, work=work, **got, **kw)
    ref = ref_norm_bwd(dy, dh, y, **kw)
    for key, t in got.items():
        if t is not None:
            assert_within(t, *ref[key], key)
