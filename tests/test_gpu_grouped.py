"""Grouped matrix products against their definition in 64 bits: ragged and
empty groups, slots and gaps, padded rows, garbage where nothing may be read,
both types, both directions and the weight gradient."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm
import moe_synth as ms
from _block_ref import assert_within, groups_of, product_bound, ref_product, ref_wgrad

pytestmark = pytest.mark.gpu

NAN = float("nan")
RAGGED = [0, 1, 15, 16, 17, 0, 63, 64, 65, 255, 256, 257, 272, 288, 289, 513, 0, 31]


def padded(shape, ld, dtype, gen, scale=1.0):
    """A [..., C] view of rows `ld` elements apart whose padding is NaN."""
    t = torch.full((*shape[:-1], ld), NAN, device="cuda", dtype=dtype)
    t[..., :shape[-1]] = scale * torch.randn(shape, generator=gen, device="cuda")
    return t[..., :shape[-1]]


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


PRODUCTS = [
    # counts, slots, gap, C, F, padding of x and w rows, dtype
    (RAGGED, 1, 0, 128, 256, 0, torch.bfloat16),
    (RAGGED, 2, 3, 200, 300, 8, torch.bfloat16),
    (RAGGED, 3, 1, 64, 64, 0, torch.float16),
    ([1], 1, 0, 8, 8, 0, torch.bfloat16),
    ([1], 1, 2, 1000, 513, 24, torch.float16),
    ([5], 1, 0, 520, 1, 0, torch.bfloat16),
    ([0, 0, 3, 0], 2, 0, 72, 136, 0, torch.bfloat16),
    ([700, 0, 2, 30], 4, 5, 136, 264, 8, torch.float16),
    ([1100], 1, 0, 320, 640, 0, torch.bfloat16),
    ([(7 * i) % 41 for i in range(1024)], 64, 0, 64, 72, 0, torch.bfloat16),
    # few rows in all
    ([1, 0, 2, 0, 1], 1, 0, 1003, 300, 8, torch.bfloat16),
    ([0, 3, 5], 1, 0, 264, 520, 0, torch.float16),
    ([2, 1], 1, 1, 4099, 77, 0, torch.bfloat16),
    ([4], 1, 0, 16384, 200, 0, torch.float16),
    ([0, 8], 1, 0, 72, 20000, 0, torch.bfloat16),
    ([1], 1, 1, 3, 5, 0, torch.bfloat16),
    ([0, 3], 1, 0, 136, 72, 0, torch.bfloat16),
    ([2], 1, 0, 136, 72, 0, torch.float16),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("case", range(len(PRODUCTS)))
def test_product(case, trans):
    counts, slots, gap, C, F, pad, dt = PRODUCTS[case]
    gen = gen_of(case)
    cnt, off, rows = groups_of(counts, slots, gap)
    G = len(counts)
    up8 = lambda n: (n + pad + 7) // 8 * 8  # noqa: E731
    x = padded((slots, rows, C), up8(C), dt, gen)
    w = padded((G, C, F) if trans else (G, F, C), up8(F if trans else C), dt, gen, 0.1)
    ref, mag, live = ref_product(x, w, cnt, off, trans)
    x.masked_fill_(~live[..., None], NAN)  # rows of no group hold anything
    out = torch.full((slots, rows, F + 3), 7.0, device="cuda", dtype=dt)[..., :F]
    sm.moe_grouped_matmul(x, w, cnt, off, out, trans_w=trans)
    torch.cuda.synchronize()
    assert_within(out[live], ref[live], mag[live], "product", product_bound(C))
    assert bool((out[~live] == 7.0).all()), "a row outside the groups was written"
    again = torch.zeros_like(out)
    sm.moe_grouped_matmul(x, w, cnt, off, again, trans_w=trans)
    assert torch.equal(again[live], out[live])


WGRADS = [
    (RAGGED, 1, 0, 128, 256, 0, torch.bfloat16),
    (RAGGED, 2, 3, 200, 304, 8, torch.bfloat16),
    (RAGGED, 3, 1, 64, 72, 0, torch.float16),
    ([1], 1, 0, 8, 8, 0, torch.bfloat16),
    ([0, 0, 3, 0], 2, 0, 1032, 136, 0, torch.float16),
    ([700, 0, 2, 30], 4, 5, 264, 520, 8, torch.bfloat16),
    ([0, 0], 1, 4, 64, 64, 0, torch.bfloat16),
    ([(7 * i) % 41 for i in range(1024)], 64, 0, 64, 72, 0, torch.bfloat16),
    # tiles of 256 columns (more than one for each pair at 128), and of 128 with long and ragged groups
    (RAGGED * 3, 2, 3, 712, 520, 8, torch.bfloat16),
    ([300, 5, 0, 77, 130, 64, 9, 16], 4, 2, 1096, 776, 0, torch.float16),
    ([2000, 1999], 1, 0, 392, 264, 0, torch.bfloat16),
    ([150, 33, 0, 401], 1, 2, 840, 136, 8, torch.float16),
]


@pytest.mark.parametrize("out_dt", ["same", "fp32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", range(len(WGRADS)))
def test_wgrad(case, accumulate, out_dt):
    counts, slots, gap, C, F, pad, dt = WGRADS[case]
    gen = gen_of(100 + case)
    cnt, off, rows = groups_of(counts, slots, gap)
    G = len(counts)
    x = padded((slots, rows, C), C + pad, dt, gen)
    dy = padded((slots, rows, F), F + pad, dt, gen, 0.3)
    ref, mag = ref_wgrad(dy, x, cnt, off)
    live = ref_product(x, torch.zeros(G, 8, C, device="cuda", dtype=dt), cnt, off, False)[2]
    x.masked_fill_(~live[..., None], NAN)
    dy.masked_fill_(~live[..., None], NAN)
    odt = dt if out_dt == "same" else torch.float32
    # odd strides take the element-wise stores
    dw = torch.randn(G, F, C + (0 if case % 2 else 3), generator=gen, device="cuda").to(odt)[..., :C]
    old = dw.double()
    if not accumulate:
        dw.fill_(NAN)
    sm.moe_grouped_wgrad(dy, x, cnt, off, dw, accumulate=accumulate)
    if accumulate:
        ref, mag = ref + old, mag + old.abs()
    assert_within(dw, ref, mag, "wgrad", product_bound(max(counts)) + 2.0 ** -23)


def test_infinite_values_stay_in_their_group():
    """An infinity in one group's rows reaches that group's results only."""
    cnt, off, rows = groups_of([20, 9, 33])
    gen = gen_of(7)
    x = torch.randn(1, rows, 64, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(1, rows, 64, generator=gen, device="cuda").bfloat16()
    w = torch.randn(3, 64, 64, generator=gen, device="cuda").bfloat16()
    x[0, 20:29], dy[0, 20:29] = float("inf"), NAN
    out, dw = torch.empty(1, rows, 64, device="cuda", dtype=torch.bfloat16), torch.empty_like(w)
    sm.moe_grouped_matmul(x, w, cnt, off, out)
    sm.moe_grouped_wgrad(dy, x, cnt, off, dw)
    assert bool(out[0, :20].isfinite().all()) and bool(out[0, 29:].isfinite().all())
    assert bool(dw[[0, 2]].isfinite().all()) and not bool(dw[1].isfinite().any())


def test_groups_outside_their_slot_are_empty_and_flagged():
    gen = gen_of(3)
    x = torch.randn(40, 64, generator=gen, device="cuda").bfloat16()
    w = torch.randn(4, 64, 64, generator=gen, device="cuda").bfloat16()
    cnt = torch.tensor([10, 31, -1, 5], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 10, 20, -3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((40, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    dw = torch.full_like(w, NAN)
    sm.moe_grouped_matmul(x, w, cnt, off, out, status=status)
    assert int(status) == sm.SYM_STATUS_OVERFLOW
    status.zero_()
    sm.moe_grouped_wgrad(x, x, cnt, off, dw, status=status)
    assert int(status) == sm.SYM_STATUS_OVERFLOW
    assert bool((out[10:] == 7.0).all()) and not bool((out[:10] == 7.0).all())
    assert bool((dw[1:] == 0).all()) and bool(dw[0].isfinite().all())


@pytest.mark.parametrize("rows,trans", [(4, False), (4, True), (9, False)])
def test_bad_groups_among_few_rows(rows, trans):
    gen = gen_of(4)
    x = torch.randn(rows, 64, generator=gen, device="cuda").bfloat16()
    w = torch.randn(3, 64, 64, generator=gen, device="cuda").bfloat16()
    cnt = torch.tensor([2, rows, -2], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((rows, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    sm.moe_grouped_matmul(x, w, cnt, off, out, trans_w=trans, status=status)
    assert int(status) == sm.SYM_STATUS_OVERFLOW
    assert bool((out[2:] == 7.0).all()) and not bool((out[:2] == 7.0).any(1).all())


TENS = [  # counts, C, F
    ([9], 7168, 2048),
    ([16], 64, 16),
    ([13], 1001, 70),
    ([0, 12, 0], 37, 1000),
    ([17, 0, 0, 15], 520, 264),
    ([1, 9, 8, 4, 10], 136, 130),
    ([3, 0, 2, 2, 1, 1, 0, 3], 328, 9),
    ([0, 0, 31, 0], 2056, 4096),
    ([10], 96, 5000),
    ([20, 0, 3, 0], 200, 5000),
    ([0] * 60 + [5, 0, 7, 1], 200, 152),
    # fewer: runs of three and four rows of a group
    ([0, 3, 0, 1], 1001, 200),
    ([4, 0, 0, 0], 136, 72),
    ([0, 0, 0, 7, 1], 264, 1000),
]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", range(len(TENS)))
def test_tens_of_rows(case, dt, trans):
    counts, C, F = TENS[case]
    gen = gen_of(300 + case)
    cnt, off, rows = groups_of(counts, 1, 0)
    G, pad = len(counts), lambda n: (n + 15) // 8 * 8  # noqa: E731
    x = torch.full((1, rows, pad(C)), NAN, device="cuda", dtype=dt)[..., :C]
    x.copy_(torch.randn(1, rows, C, generator=gen, device="cuda"))
    w = torch.full((G, C, pad(F)) if trans else (G, F, pad(C)), NAN, device="cuda", dtype=dt)[..., :F if trans else C]
    w.copy_(0.05 * torch.randn(w.shape, generator=gen, device="cuda"))
    wide = torch.full((1, rows, F + 3), 7.0, device="cuda", dtype=dt)
    out = wide[..., :F]
    out.fill_(NAN)
    sm.moe_grouped_matmul(x, w, cnt, off, out, trans_w=trans)
    ref, mag, _ = ref_product(x, w, cnt, off, trans)
    assert_within(out, ref, mag, "product", product_bound(C))
    assert bool((wide[..., F:] == 7.0).all())
    again = torch.empty_like(wide)[..., :F]
    sm.moe_grouped_matmul(x, w, cnt, off, again, trans_w=trans)
    assert torch.equal(out, again)


@pytest.mark.parametrize("trans", [False, True])
def test_bad_groups_and_infinities_among_tens_of_rows(trans):
    gen = gen_of(6)
    x = torch.randn(15, 64, generator=gen, device="cuda").bfloat16()
    x[4] = float("inf")
    w = torch.randn(4, 64, 64, generator=gen, device="cuda").bfloat16()
    cnt = torch.tensor([4, 15, -2, 5], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 1, 3, 5], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((15, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    sm.moe_grouped_matmul(x, w, cnt, off, out, trans_w=trans, status=status)
    assert int(status) == sm.SYM_STATUS_OVERFLOW
    assert bool((out[[4] + list(range(10, 15))] == 7.0).all()) and bool(out.isfinite().all())
    assert not bool((out[:4] == 7.0).any(1).all()) and not bool((out[5:10] == 7.0).any(1).all())


def test_empty_tensors():
    cnt = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(2, 64, 64, device="cuda", dtype=torch.bfloat16)
    sm.moe_grouped_matmul(x, w, cnt, cnt, x)
    sm.moe_grouped_wgrad(x, x, cnt, cnt, w)
    assert bool((w == 0).all())


def test_rows_past_32_bit_element_offsets():
    """Groups at the end of tensors of more than 2^32 elements."""
    rows, C, F = 300_000, 16384, 16384
    x = torch.empty(rows, C, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(rows, F, device="cuda", dtype=torch.bfloat16)
    n = 37
    gen = gen_of(11)
    x[-n:] = torch.randn(n, C, generator=gen, device="cuda")
    w = (0.02 * torch.randn(1, F, C, generator=gen, device="cuda")).bfloat16()
    cnt = torch.tensor([n], dtype=torch.int32, device="cuda")
    off = torch.tensor([rows - n], dtype=torch.int32, device="cuda")
    sm.moe_grouped_matmul(x, w, cnt, off, out)
    ref, mag, _ = ref_product(x[None, -n:], w, cnt[None], torch.zeros_like(cnt)[None], False)
    assert_within(out[-n:], ref[0], mag[0], "product", product_bound(C))
    dw = torch.empty(1, F, C, device="cuda", dtype=torch.bfloat16)
    out[-n:] = torch.randn(n, F, generator=gen, device="cuda")
    sm.moe_grouped_wgrad(out, x, cnt, off, dw)
    ref, mag = ref_wgrad(out[None, -n:], x[None, -n:], cnt[None], torch.zeros_like(cnt)[None])
    assert_within(dw, ref, mag, "wgrad", product_bound(n))


def test_long_groups_and_wide_contractions():
    """Many K blocks on both sides: 5000 rows, 4104 columns."""
    counts, C, F = [5000, 3], 4104, 520
    gen = gen_of(5)
    cnt, off, rows = groups_of(counts)
    x = torch.randn(1, rows, C, generator=gen, device="cuda").bfloat16()
    w = (0.02 * torch.randn(2, F, C, generator=gen, device="cuda")).bfloat16()
    out = torch.empty(1, rows, F, device="cuda", dtype=torch.bfloat16)
    sm.moe_grouped_matmul(x, w, cnt, off, out)
    ref, mag, _ = ref_product(x, w, cnt, off, False)
    assert_within(out, ref, mag, "product", product_bound(C))
    dw = torch.empty(2, F, C, device="cuda", dtype=torch.float32)
    sm.moe_grouped_wgrad(out, x, cnt, off, dw)
    ref, mag = ref_wgrad(out, x, cnt, off)
    assert_within(dw, ref, mag, "wgrad", product_bound(5000))


def test_on_a_side_stream():
    gen = gen_of(9)
    cnt, off, rows = groups_of([200, 100])
    x = torch.randn(1, rows, 256, generator=gen, device="cuda").bfloat16()
    w = torch.randn(2, 256, 256, generator=gen, device="cuda").bfloat16()
    want = torch.empty(1, rows, 256, device="cuda", dtype=torch.bfloat16)
    sm.moe_grouped_matmul(x, w, cnt, off, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [torch.empty_like(want) for _ in range(8)]
    for i, t in enumerate(got):  # calls on two streams share nothing
        sm.moe_grouped_matmul(x, w, cnt, off, t, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got)


def test_on_a_heap_the_products_are_the_expert_ffn():
    """gate, up, SwiGLU and down over a heap's windows against the fused FFN's y."""
    cfg = dict(world=2, tokens_per_slot=200, hidden=256, num_experts=4, topk=2, inter=384)
    dev = torch.device("cuda")
    x = ms.x_torch(cfg, dev)
    wg, wu, wd = ms.weights_torch(cfg, dev)
    n = 400
    heap = sm.SymHeap(cfg, dev)
    idx = torch.empty(n, 2, dtype=torch.int32, device=dev)
    w = torch.empty(n, 2, device=dev)
    heap.route_topk(ms.logits_torch(cfg, dev), idx, w)
    heap.dispatch(x, idx, w)
    heap.expert_ffn(wg, wu, wd)
    torch.cuda.synchronize()
    win = heap.window
    y_ref, h_ref = win("y").clone(), win("h").clone()
    shape = (2, heap.cap, 384)
    g, u = (torch.empty(shape, device=dev, dtype=torch.bfloat16) for _ in range(2))
    groups = dict(cnt=win("cnt"), off=win("recv_off"), status=heap.status_word())
    view = lambda t: t.view(4, *t.shape[-2:])  # noqa: E731
    sm.moe_grouped_matmul(win("recv_x"), view(wg), out=g, **groups)
    sm.moe_grouped_matmul(win("recv_x"), view(wu), out=u, **groups)
    win("h").zero_(), win("y").zero_()
    sm.moe_swiglu_rows(g, u, win("h"), total=win("total"))
    sm.moe_grouped_matmul(win("h"), view(wd), out=win("y"), **groups)
    assert heap.status() == 0
    for d in range(2):
        t = int(win("total")[d])
        # the fused path rounds h once, this one g and u before it: three
        # roundings to 8 bits against one
        torch.testing.assert_close(win("h")[d, :t].float(), h_ref[d, :t].float(), rtol=3 * 2.0 ** -8, atol=1e-3)
        rel = (win("y")[d, :t].float() - y_ref[d, :t].float()).norm() / y_ref[d, :t].float().norm()
        assert float(rel) < 1e-2


def _args(**over):
    a = dict(x=torch.zeros(16, 64, device="cuda", dtype=torch.bfloat16),
             w=torch.zeros(2, 64, 64, device="cuda", dtype=torch.bfloat16),
             cnt=torch.zeros(2, dtype=torch.int32, device="cuda"), off=torch.zeros(2, dtype=torch.int32, device="cuda"),
             out=torch.zeros(16, 64, device="cuda", dtype=torch.bfloat16))
    a.update(over)
    return a


@pytest.mark.parametrize("bad", [
    dict(x=torch.zeros(16, 64, dtype=torch.bfloat16)),                                # not on the device
    dict(out=torch.zeros(15, 64, dtype=torch.bfloat16)),                              # rows differ
    dict(out=torch.zeros(16, 64, dtype=torch.float32)),                               # types differ
    dict(w=torch.zeros(2, 64, 72, dtype=torch.bfloat16)),                             # C differs
    dict(w=torch.zeros(3, 64, 64, dtype=torch.bfloat16)),                             # E differs
    dict(w=torch.zeros(2, 64, 64, dtype=torch.bfloat16).transpose(1, 2)),             # inner stride
    dict(cnt=torch.zeros(2, dtype=torch.int64)),                                      # not int32
    dict(off=torch.zeros(3, dtype=torch.int32)),
    dict(x=torch.zeros(16, 65, dtype=torch.bfloat16)[:, :64]),                        # row stride no multiple of 8
    dict(x=torch.zeros(16 * 64 + 4, dtype=torch.bfloat16)[4:].view(16, 64)),          # base not 16-byte aligned
    dict(x=torch.zeros(1, 64, dtype=torch.bfloat16).expand(16, 64)),                  # rows overlap
    dict(x=torch.zeros(16, 64), w=torch.zeros(2, 64, 64), out=torch.zeros(16, 64)),   # fp32 operands
    dict(w=torch.zeros(1, 64, 64, dtype=torch.bfloat16).expand(2, 64, 64)),           # one matrix for two groups
])
def test_refusals(bad):
    device = lambda k, t: t if k == "x" and tuple(t.shape) == (16, 64) and t.dtype == torch.bfloat16 and t.is_contiguous() \
        and t.data_ptr() % 16 == 0 else None  # noqa: E731
    moved = {}
    for k, t in bad.items():
        if device(k, t) is not None:
            moved[k] = t  # the one that stays on the host
            continue
        room = torch.zeros(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype, device="cuda")
        moved[k] = room.as_strided(t.size(), t.stride(), t.storage_offset())
    with pytest.raises(sm.SymmoeError) as ei:
        sm.moe_grouped_matmul(**_args(**moved))
    assert ei.value.code == sm.SYM_EINVAL
