"""Block norms between 4096 and 6144 columns, where the forward of 16-bit types
runs two blocks an SM with a layout of its own: shared gates, a gate for each
row, with and without dropout, and blocks that walk many rows."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import assert_within, ref_norm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("rows,gates", [(3, 1), (1300, 1), (1302, 6), (700, 700), (700, 350), (610, 0)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cols", [4104, 5120, 6144])
def test_forward(cols, dt, rows, gates, p):
    gen = torch.Generator(device="cuda").manual_seed(cols + rows)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    x, o, w_post, w_pre = randn(rows, cols), randn(rows, cols), (1 + 0.2 * randn(cols)).to(dt), (1 + 0.2 * randn(cols)).to(dt)
    kw = dict(o=o, w_post=w_post, w_pre=w_pre, gate=randn(gates, cols) if gates else None, gate_act="tanh" if gates else "none",
              scale=0.6, p=p, seed=5, offset=6)
    out = dict(y=torch.empty_like(x), h=torch.empty_like(x), rstd_post=torch.empty(rows, device="cuda"),
               rstd_pre=torch.empty(rows, device="cuda"))
    sm.moe_block_norm(x, **out, **kw)
    ref, mag = ref_norm(x, **kw)
    assert_within(out["y"], ref["y"], mag["y"], "y")
    assert_within(out["h"], ref["h"], mag["h"] + ref["h"].abs(), "h")
    assert_within(out["rstd_post"], ref["rstd_post"], ref["rstd_post"], "rstd_post")
    assert_within(out["rstd_pre"], ref["rstd_pre"], ref["rstd_pre"], "rstd_pre")
    again = torch.empty_like(x)
    sm.moe_block_norm(x, y=again, **{k: v for k, v in kw.items() if k != "w_pre"})
    assert torch.equal(again, out["y"])
