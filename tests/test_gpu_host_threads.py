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
