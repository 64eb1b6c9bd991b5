"""The whole MoE layer for a few tokens against its definition in 64 bits."""
import math

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _more_ref import ref_few_tokens, ref_route

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


class Layer:
    def __init__(self, T, H, I, E, k, dt=BF, fused=False, pad=0, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dt)
        self.k, self.dt = k, dt
        self.x = rand(T, H + pad)[:, :H]
        if fused:
            both = rand(E, 2 * I + 3, H + pad, scale=H ** -0.5)
            self.wg, self.wu = both[:, :I, :H], both[:, I:2 * I, :H]
        else:
            self.wg, self.wu = rand(E, I, H + pad, scale=H ** -0.5)[..., :H], rand(E, I, H + pad, scale=H ** -0.5)[..., :H]
        self.wd = rand(E, H, I + pad, scale=I ** -0.5)[..., :I]
        self.wr = rand(E, H + pad, scale=H ** -0.5)[:, :H]
        self.logits = torch.randn(T, E, generator=gen, device="cuda")

    def call(self, router=False, out=None, work=None):
        T, H = self.x.shape
        idx = torch.full((T, self.k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, self.k), -7.0, device="cuda")
        out = torch.full((T, H), 7.0, device="cuda", dtype=self.dt) if out is None else out
        logits = torch.full_like(self.logits, 7.0) if router else self.logits
        n = sm.moe_few_tokens_workspace(T, self.wg.shape[1], self.k)
        work = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) if work is None else work
        sm.moe_few_tokens(self.x, self.wg, self.wu, self.wd, logits, idx, w, out, work, w_router=self.wr if router else None)
        return logits, idx, w, out

    def check(self, router=False):
        logits, idx, w, out = self.call(router)
        if router:
            ref = self.x.double() @ self.wr.double().T
            mag = self.x.double().abs() @ self.wr.double().abs().T
            assert bool(((logits.double() - ref).abs() <= 1e-5 * mag).all())
        want, weights = ref_route(logits, self.k)
        assert idx.tolist() == want
        got = w.double().cpu()
        ref_w = torch.tensor(weights, dtype=torch.float64).reshape(got.shape)
        assert bool(((got - ref_w).abs() <= 2e-6 * ref_w).all())
        dead = [[float(logits[t, e]) == -math.inf for e in row] for t, row in enumerate(want)]
        ref, bound = ref_few_tokens(self.x, self.wg, self.wu, self.wd, want, weights, dead)
        err = (out.double() - ref).abs()
        assert bool((err <= bound).all()), (float((err / bound).max()), int((err > bound).sum()))
        return out


#         T   H     I    E   k
SIZES = [(1, 8, 8, 1, 1), (1, 128, 256, 4, 2), (2, 64, 8, 3, 3), (3, 8, 72, 5, 2), (4, 136, 264, 4, 2), (5, 1032, 520, 24, 3),
         (7, 520, 1032, 9, 4), (8, 512, 512, 8, 2), (9, 256, 512, 1, 1), (16, 640, 384, 2, 2), (17, 264, 136, 3, 2),
         (32, 256, 256, 4, 1), (32, 512, 128, 256, 8), (32, 128, 128, 1, 1), (31, 136, 200, 2, 1), (6, 2048, 1408, 60, 6),
         (1, 4096, 1544, 8, 2), (2, 7168, 264, 33, 32), (32, 1096, 72, 40, 32), (1, 72, 4104, 1024, 4),
         (32, 72, 40, 1024, 32), (3, 16384, 24, 2, 1)]


@pytest.mark.parametrize("T,H,I,E,k", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("router", [False, True])
def test_sizes(T, H, I, E, k, dt, router):
    Layer(T, H, I, E, k, dt, fused=router).check(router)


@pytest.mark.parametrize("pad", [8, 24, 64])
@pytest.mark.parametrize("fused", [False, True])
def test_strides(pad, fused):
    layer = Layer(6, 264, 520, 5, 2, BF, fused, pad)
    out = torch.full((6, 264 + pad + 1), 7.0, device="cuda", dtype=BF)
    want = layer.check(True)
    layer.call(True, out=out[:, 1:265])  # an output of any stride, off every alignment
    assert torch.equal(out[:, 1:265], want)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 265:] == 7).all())


@pytest.mark.parametrize("T", [1, 8, 9, 16, 17, 24, 25, 32])
def test_all_tokens_on_one_expert(T):
    layer = Layer(T, 264, 264, 6, 2)
    layer.logits[:, 4] = 9.0
    layer.logits[:, 1] = 8.0
    layer.check()


def test_ties_go_to_the_lower_expert():
    layer = Layer(5, 64, 64, 40, 6)
    layer.logits.zero_()
    layer.logits[2, 33:] = 1.0
    layer.logits[3, ::7] = 2.0
    layer.logits[4] = -0.0
    layer.logits[4, 5] = 0.0
    layer.check()
    idx = layer.call()[1].tolist()
    assert idx[0] == [0, 1, 2, 3, 4, 5] and idx[2] == [33, 34, 35, 36, 37, 38] and idx[3] == [0, 7, 14, 21, 28, 35]
    assert idx[4] == [0, 1, 2, 3, 4, 5]


def test_masked_experts():
    """Experts masked with -inf take no part: one left, none left, the lowest finite value beside them."""
    layer = Layer(5, 136, 72, 8, 3)
    inf = math.inf
    layer.logits[0, 1:] = -inf
    layer.logits[1, :] = -inf
    layer.logits[2, :6] = -inf
    layer.logits[3, :] = torch.finfo(torch.float32).min
    layer.logits[4, 2:] = torch.finfo(torch.float32).min
    out = layer.check()
    assert not out[1].any()
    # what a masked expert holds is not read into the result
    layer.logits[:, 5] = -inf
    clean = layer.check()
    for w in (layer.wg, layer.wu, layer.wd):
        w[5] = float("nan")
    assert torch.equal(layer.call()[3], clean)


def test_infinite_and_nan_logits_stay_in_their_row():
    layer = Layer(6, 64, 72, 5, 2)
    clean = layer.call()
    layer.logits[1, 3] = math.inf
    layer.logits[3, :] = math.nan
    layer.logits[4, :4] = math.nan  # one number left, so a NaN is chosen beside it
    logits, idx, w, out = layer.call()
    for t in (1, 3, 4):
        assert bool(out[t].isnan().all()) and bool(w[t].isnan().any())
    assert idx[1, 0] == 3 and idx[3].tolist() == [0, 1] and idx[4].tolist() == [4, 0]
    for t in (0, 2, 5):
        assert torch.equal(out[t], clean[3][t]) and torch.equal(idx[t], clean[1][t])
    # a NaN that is not chosen does not matter
    layer = Layer(2, 64, 72, 5, 2)
    layer.logits[0, int(layer.logits[0].argmin())] = math.nan
    layer.check()


def test_infinities_in_a_token_stay_in_its_row():
    layer = Layer(9, 136, 72, 2, 2)
    clean = layer.call()[3]
    layer.x[4, 7] = math.inf
    layer.x[6, 0] = math.nan
    out = layer.call()[3]
    rest = [t for t in range(9) if t not in (4, 6)]
    assert torch.equal(out[rest], clean[rest])
    assert bool(out[6].isnan().all()) and not bool(out[4].isfinite().all())


def test_in_place_capture_and_order():
    layer = Layer(8, 520, 264, 12, 3)
    want = layer.call(True)
    work = torch.empty(sm.moe_few_tokens_workspace(8, 264, 3), dtype=torch.uint8, device="cuda")
    keep = layer.x.clone()
    layer.x = keep.clone()
    assert torch.equal(layer.call(True, out=layer.x)[3], want[3])  # out is x
    layer.x = keep
    idx, w, out = torch.empty_like(want[1]), torch.empty_like(want[2]), torch.empty_like(want[3])
    logits = torch.empty_like(layer.logits)
    go = lambda: sm.moe_few_tokens(layer.x, layer.wg, layer.wu, layer.wd, logits, idx, w, out, work, w_router=layer.wr)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go()
        with torch.cuda.graph(graph, stream=side):
            go()  # two layers one after another, sharing a workspace
            go()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for t in (idx, w, out, logits):
            t.fill_(7)
        work.fill_(255)
        graph.replay()
        assert torch.equal(out, want[3]) and torch.equal(idx, want[1]) and torch.equal(w, want[2]) and torch.equal(logits, want[0])
    # a layer's output is the next one's input, and weights change between calls, with nothing waited for
    chain = layer.x.clone()
    for _ in range(4):
        layer.x = chain
        chain = layer.call(True)[3]
        layer.wd.mul_(1.0)
    torch.cuda.synchronize()
    ref = keep.clone()
    for _ in range(4):
        layer.x = ref
        ref = layer.call(True)[3]
        torch.cuda.synchronize()
    assert torch.equal(chain, ref)


def test_same_rows_as_the_pipeline():
    """The heap's pipeline on the same tokens: it rounds h and every expert's row to bf16, nothing else differs."""
    shape = dict(world=2, tokens_per_slot=16, hidden=256, inter=384, num_experts=8, topk=2)
    layer = Layer(32, 256, 384, 8, 2)
    heap = sm.SymHeap(shape, "cuda")
    idx, w, out = torch.empty(32, 2, dtype=torch.int32, device="cuda"), torch.empty(32, 2, device="cuda"), torch.empty(32, 256, device="cuda", dtype=BF)
    heap.pipeline(layer.logits, layer.x.contiguous(), layer.wg.contiguous(), layer.wu.contiguous(), layer.wd.contiguous(), idx, w, out)
    _, idx2, w2, out2 = layer.call()
    assert torch.equal(idx, idx2)
    assert float((w - w2).abs().max()) <= 2e-6
    # h's and y's roundings of 2^-8 each, taken at their worst against sums of absolute values
    e, h64 = idx.long(), lambda a, x: (a.double() @ x.double().unsqueeze(2)).squeeze(2)
    mag = torch.zeros(32, 256, dtype=torch.float64, device="cuda")
    for j in range(2):
        g, u = h64(layer.wg[e[:, j]], layer.x), h64(layer.wu[e[:, j]], layer.x)
        hj = (g * torch.sigmoid(g) * u).abs()
        mag += w[:, j:j + 1].double() * h64(layer.wd[e[:, j]].abs(), hj)
    assert bool(((out.double() - out2.double()).abs() <= 2.0 ** -8 * (2 * mag + out.double().abs() + out2.double().abs()) * 1.01).all())


def test_no_tokens():
    layer = Layer(1, 64, 64, 4, 2)
    layer.x, layer.logits = layer.x[:0], layer.logits[:0]
    layer.call()


def test_refusals():
    layer = Layer(4, 64, 72, 6, 2)
    T, k = 4, 2
    idx, w, out = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty_like(layer.x)
    work = torch.empty(sm.moe_few_tokens_workspace(T, 72, k), dtype=torch.uint8, device="cuda")
    good = dict(x=layer.x, w_gate=layer.wg, w_up=layer.wu, w_down=layer.wd, logits=layer.logits, idx=idx, w=w, out=out, work=work,
                w_router=layer.wr)
    sm.moe_few_tokens(**good)
    many = torch.zeros(33, 64, device="cuda", dtype=BF)
    bad = [dict(x=layer.x.half()), dict(x=layer.x[:3]), dict(x=layer.x.cpu()), dict(x=layer.x[0]), dict(w_gate=layer.wg[:5]),
           dict(w_up=layer.wu[:, :64]), dict(w_down=layer.wg), dict(w_down=layer.wd.half()), dict(w_gate=layer.wg.transpose(1, 2)),
           dict(logits=layer.logits.half()), dict(logits=layer.logits.t().contiguous().t()), dict(idx=idx.long()), dict(idx=idx[:3]),
           dict(w=w[:, :1]), dict(w=w.double()), dict(out=out.float()), dict(out=out[:, :32]), dict(w_router=layer.wr[:5]),
           dict(work=work.cpu()), dict(work=None), dict(w=None),
           dict(x=many, out=many.clone(), logits=torch.zeros(33, 6, device="cuda"), idx=idx.new_empty(33, k), w=w.new_empty(33, k)),
           dict(idx=idx.new_empty(T, 7), w=w.new_empty(T, 7))]
    for i, kw in enumerate(bad):
        with pytest.raises(sm.SymmoeError) as e:
            sm.moe_few_tokens(**dict(good, **kw))
        assert e.value.code == sm.SYM_EINVAL, i
    with pytest.raises(sm.SymmoeError) as e:
        sm.moe_few_tokens(**dict(good, work=work[:work.numel() - 16]))
    assert e.value.code == sm.SYM_ENOSPACE
