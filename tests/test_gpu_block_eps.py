"""Block norms with eps = 0, with and without a block output, in rows of every
kernel: short and long vectors, off 16-byte boundaries, beyond 8192 columns."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import assert_within, ref_norm

pytestmark = pytest.mark.gpu

COLS = [8, 256, 4096, 5120, 7168, 333, 4095, 9000, 9001]


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("has_o", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("cols", COLS)
def test_no_eps(cols, dt, has_o, p):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    x, w = randn(5, cols), (1 + 0.2 * randn(cols)).to(dt)
    # without a block output the dropout has nothing to drop
    kw = dict(o=randn(5, cols) if has_o else None, w_pre=w, p=p, seed=3, offset=4, eps=0.0)
    h, ry = torch.empty_like(x), torch.empty(5, device="cuda")
    y = torch.empty_like(x) if has_o else None
    sm.moe_block_norm(x, y=y, h=h, rstd_pre=ry, **kw)
    ref, mag = ref_norm(x, **kw)
    assert_within(h, ref["h"], mag["h"] + ref["h"].abs(), "h")
    assert_within(ry, ref["rstd_pre"], ref["rstd_pre"], "rstd_pre")
    if has_o:
        assert_within(y, ref["y"], mag["y"], "y")
