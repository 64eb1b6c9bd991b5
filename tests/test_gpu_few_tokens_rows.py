"""Rows of the few-token layer: no further from the definition in 64 bits than their own
rounding and a little puts them, whatever the sizes of what goes between the products."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


class Layer:
    def __init__(self, T, H, I, E, k, dt, x=1.0, down=None, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dt)
        self.x, self.wg, self.wu = rand(T, H, scale=x), rand(E, I, H, scale=H ** -0.5), rand(E, I, H, scale=H ** -0.5)
        self.wd, self.logits, self.k = rand(E, H, I, scale=I ** -0.5 if down is None else down), torch.randn(T, E, generator=gen, device="cuda"), k

    def call(self):
        T, H = self.x.shape
        idx, w = torch.empty(T, self.k, dtype=torch.int32, device="cuda"), torch.empty(T, self.k, device="cuda")
        out = torch.full((T, H), 7.0, device="cuda", dtype=self.x.dtype)
        work = torch.empty(sm.moe_few_tokens_workspace(T, self.wg.shape[1], self.k), dtype=torch.uint8, device="cuda").fill_(255)
        sm.moe_few_tokens(self.x, self.wg, self.wu, self.wd, self.logits, idx, w, out, work)
        return idx, w, out

    def check(self):
        """The squares of the row's rounding and of all else add up, which are independent.  All
        else is worth 0.45 of a rounding at most, 1.1 of it together: h is held to 2^-16 (fp16: 2^-22, or
        2^-36 where it is smaller), a thousandth to a hundredth of a rounding; a warp's sums of an eighth of K
        terms, at most 2048, drop 2^-24 of themselves at each 16 of them, 8e-6 where fp16
        rounds by 2e-4; the rest is fp32's."""
        idx, w, out = self.call()
        ref = torch.zeros(self.x.shape, dtype=torch.float64, device="cuda")
        for t in range(len(ref)):
            x = self.x[t].double()
            for j in range(self.k):
                e = int(idx[t, j])
                g = self.wg[e].double() @ x
                ref[t] += w[t, j].double() * (self.wd[e].double() @ (g * torch.sigmoid(g) * (self.wu[e].double() @ x)))
        norm = lambda v: torch.linalg.vector_norm(v, dim=1)
        rounding = norm(ref.to(out.dtype).double() - ref)
        err = norm(out.double() - ref)
        assert bool((err <= 1.1 * rounding).all()), (float((err / rounding).max()), float((rounding / norm(ref)).max()))


@pytest.mark.parametrize("T,H,I,E,k", [(4, 256, 512, 4, 2), (20, 520, 264, 3, 2)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("x", [0.1, 0.03, 0.01, 0.003, 0.001])
def test_small_values_between_the_products(T, H, I, E, k, dt, x):
    """h far below one, down to what fp16 cannot hold; down weights that bring the rows back up."""
    Layer(T, H, I, E, k, dt, x, down=min(100.0, x ** -1.5)).check()


# long contractions (the most slices, the deepest pipelines), many experts a token, blocks that share experts, odd slices
SIZES = [(1, 4096, 1544, 8, 2), (3, 16384, 24, 2, 1), (1, 24, 16384, 2, 2), (2, 7168, 264, 33, 32), (6, 2048, 1408, 60, 6), (5, 1032, 520, 24, 3),
         (9, 520, 1032, 9, 4), (32, 1096, 72, 40, 32), (1, 72, 4104, 1024, 4), (32, 512, 4096, 4, 2), (17, 264, 136, 3, 2), (2, 14336, 512, 4, 2),
         (1, 128, 2048, 64, 8), (32, 7168, 2048, 16, 2)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
def test_rows_are_off_by_their_rounding(T, H, I, E, k, dt):
    Layer(T, H, I, E, k, dt).check()


@pytest.mark.parametrize("dt", [BF, HF])
def test_where_the_high_parts_cancel(dt):
    """Down weights of -1 and 1 over two features whose h differ by an eighth of the high part's last
    place: what is left is the low parts' difference (a power of two, so it is exact)."""
    T, H, I = 1, 64, 64
    layer = Layer(T, H, I, 1, 1, dt)
    layer.x.zero_()
    layer.x[0, 0], layer.x[0, 1] = 8.0, 1.0
    layer.wg.zero_(), layer.wu.zero_(), layer.wd.zero_()
    layer.wg[0, :2, 0] = 4.0  # silu(32): 32 to fp32's last place
    layer.wu[0, 0, 0] = layer.wu[0, 1, 0] = 1.0 / 8
    step = 2.0 ** -7 if dt == BF else 2.0 ** -10  # hi's last place, of 1
    layer.wu[0, 1, 1] = step / 8
    layer.wd[0, :, 0], layer.wd[0, :, 1] = -1.0, 1.0
    out = layer.call()[2].double()
    want = 32 * step / 8
    assert bool(((out - want).abs() <= want * 2.0 ** -12).all()), (out[0, :4].tolist(), want)
