"""Calls from host threads other than the one that set the device up."""
import threading

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
import moe_synth as ms

pytestmark = pytest.mark.gpu


class Recorder:
    """The library; the last call's function and arguments are kept."""

    def __init__(self, lib):
        self.lib, self.last = lib, None

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*args):
            if name != "sym_strerror":
                self.last = fn, args
            return fn(*args)

        return call


def recorded(call):
    """The C call that `call` ends in, as (function, arguments)."""
    rec, lib = Recorder(sm.lib()), sm._lib
    sm._lib = rec
    try:
        call()
    finally:
        sm._lib = lib
    return rec.last


def product(counts, C, F, trans):
    gen = torch.Generator(device="cuda").manual_seed(C)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    off = (torch.cumsum(cnt, 0) - cnt).to(torch.int32)
    x = torch.randn(sum(counts), C, generator=gen, device="cuda").bfloat16()
    w = torch.randn((len(counts), C, F) if trans else (len(counts), F, C), generator=gen, device="cuda").bfloat16()
    out = torch.empty(sum(counts), F, device="cuda", dtype=torch.bfloat16)
    return lambda: sm.moe_grouped_matmul(x, w, cnt, off, out, trans_w=trans), (out, x, w, cnt, off)


def wgrad(counts, C, F):
    _, (_, x, _, cnt, off) = product(counts, C, 8, False)
    dy = torch.randn(len(x), F, generator=torch.Generator(device="cuda").manual_seed(F), device="cuda").bfloat16()
    dw = torch.empty(len(counts), F, C, device="cuda", dtype=torch.bfloat16)
    return lambda: sm.moe_grouped_wgrad(dy, x, cnt, off, dw), (dw, x, dy, cnt, off)


def ffn():
    cfg, dev = ms.CONFIGS["tiny"], torch.device("cuda")
    heap, n = sm.SymHeap(cfg, dev), cfg["world"] * cfg["tokens_per_slot"]
    idx, w = torch.empty(n, cfg["topk"], dtype=torch.int32, device=dev), torch.empty(n, cfg["topk"], device=dev)
    weights = ms.weights_torch(cfg, dev)
    heap.route_topk(ms.logits_torch(cfg, dev), idx, w)
    heap.dispatch(ms.x_torch(cfg, dev), idx, w)
    return lambda: heap.expert_ffn(*weights), (heap.window("h"), heap, idx, w, weights)


def norm(rows, cols, dt):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, o = (torch.randn(rows, cols, generator=gen, device="cuda").to(dt) for _ in range(2))
    y, h = torch.empty_like(x), torch.empty_like(x)
    return lambda: sm.moe_block_norm(x, o=o, y=y, h=h, p=0.1, seed=1), (y, h, x, o)


def norm_bwd(rows, cols, dt):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    dy, o = (torch.randn(rows, cols, generator=gen, device="cuda").to(dt) for _ in range(2))
    ro = o.double().square().mean(1).rsqrt().float()
    do = torch.empty_like(o)
    work = torch.empty(sm.moe_block_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return lambda: sm.moe_block_norm_bwd(dy=dy, o=o, rstd_post=ro, do=do, p=0.1, seed=1, work=work), (do, dy, o, ro, work)


BF16, FP32 = torch.bfloat16, torch.float32
# two sizes that take different amounts of shared memory of the same kernel
SIZES = {
    "vectors": (norm, (2, 8192, FP32), (2, 2056, FP32)),
    "vectors, gradient": (norm_bwd, (2, 8192, FP32), (2, 2056, FP32)),
    "off boundaries": (norm, (2, 8191, FP32), (2, 33, FP32)),
    "off boundaries, gradient": (norm_bwd, (2, 8191, FP32), (2, 33, FP32)),
    "long rows": (norm, (2, 65535, BF16), (2, 8201, BF16)),
    "long rows, gradient": (norm_bwd, (2, 65535, BF16), (2, 8201, BF16)),
    "few rows": (product, ([1, 1, 1, 1], 16384, 64, True), ([1], 64, 64, True)),
    "tens of rows": (product, ([12, 0, 10, 9], 256, 64, False), ([9, 0, 0, 0], 256, 64, False)),
    "many rows": (product, ([1] * 1000, 64, 64, False), ([100], 64, 64, False)),
}


@pytest.mark.parametrize("name", SIZES)
def test_threads_with_different_sizes(name):
    """Six threads at once, each on a stream and outputs of its own: a call that sets
    a kernel up for its size must not undo what another one has just set up."""
    make, *sizes = SIZES[name]
    made = [make(*sizes[i % 2]) for i in range(6)]
    calls = [recorded(call) for call, _ in made]
    torch.cuda.synchronize()
    outs = [kept[0] for _, kept in made]
    want = [t.clone() for t in outs]
    streams = [torch.cuda.Stream() for _ in made]
    for t in outs:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    start, codes = threading.Barrier(len(made)), [set() for _ in made]

    def work(i):
        (fn, args), handle = calls[i], streams[i].cuda_stream
        args = (*args[:-1], handle)
        start.wait()
        for _ in range(3000):
            codes[i].add(fn(*args))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{sm.SYM_OK}] * len(made)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("make", [lambda: product([100, 3], 64, 64, False), lambda: product([1], 64, 64, True),
                                  lambda: wgrad([100, 3], 64, 64), ffn],
                         ids=["product", "product of one row", "weight gradient", "expert ffn"])
def test_a_thread_without_a_context(make):
    """The C call as the first CUDA call of its thread."""
    call, (out, *_keep) = make()
    fn, args = recorded(call)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    codes = []
    t = threading.Thread(target=lambda: codes.append(fn(*args)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert codes == [sm.SYM_OK]
    assert torch.equal(out, want)
