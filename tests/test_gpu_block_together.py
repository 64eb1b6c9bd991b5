"""The layer norm, the layer for a few tokens and the orthogonalised updates as they
are used: a trained block answering tokens, its update from its own gradients, and
both in one captured step."""
import importlib.util
import os

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
import moe_synth as ms
from _block_ref import UNIT
from _more_ref import ref_few_tokens, ref_layer_norm, ref_orthogonalize, ref_route

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_moe_block", os.path.join(ROOT, "examples", "train_moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def config(**kw):
    return dict(ms.shape_of(ms.CONFIGS["tiny"]), **kw)


@pytest.mark.parametrize("tokens", [1, 5, 32])
def test_the_trained_block_answers_as_its_forward(tokens):
    """The same block through the heap and by itself: the same experts; what differs
    are h, the experts' rows and the combine's sum, rounded on the heap's way."""
    ex = example()
    cfg = config(tokens_per_slot=16)
    block = ex.MoeBlock(cfg, dropout=0.0)
    x = ms.x_torch(cfg, torch.device("cuda"))
    y, few = torch.empty_like(x), torch.empty(tokens, x.shape[1], device="cuda", dtype=BF)
    block.forward(x, y)
    block.answer(x[:tokens].contiguous(), few)
    # Errors of 2^-8 in h, in an expert's row and in the layer's output, each of at most the
    # sum of the terms' absolute values, go through a norm (twice: numerator and length) and
    # a gate of tanh(0.5) times scale; both results are then rounded.
    out = block.out[:tokens].double()
    rms = out.square().mean(1, keepdim=True).sqrt()
    q, I = block.params, cfg["inter"]
    mag = torch.zeros_like(out)
    for j in range(block.k):
        e = block.idx[:tokens, j].long()
        h64 = block.h[:tokens].double()
        g = torch.einsum("tih,th->ti", q["gate_up"][e, :I].double(), h64)
        u = torch.einsum("tih,th->ti", q["gate_up"][e, I:].double(), h64)
        act = (g * torch.sigmoid(g) * u).abs()
        mag += block.w[:tokens, j:j + 1].double() * torch.einsum("thi,ti->th", q["down"][e].double().abs(), act)
    d = 2.0 ** -8 * 3 * mag  # of the layer's output
    slack = 0.5 * 0.4622 * (d + out.abs() / rms * d.square().mean(1, keepdim=True).sqrt()) / rms * 1.05
    bound = slack + UNIT[BF] * (few.double().abs() + y[:tokens].double().abs()) + 1e-6
    assert bool(((few.double() - y[:tokens].double()).abs() <= bound).all())


def test_orthogonal_update_of_the_examples_gradients():
    """The update that the example makes is the definition's of its own weight gradients."""
    ex = example()
    cfg = config(tokens_per_slot=16)
    block = ex.MoeBlock(cfg, dropout=0.0)
    x = ms.x_torch(cfg, torch.device("cuda"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    block.forward(x, y)
    block.backward(x, dx)
    before = {k: t.clone() for k, t in block.params.items()}
    I, lr = cfg["inter"], 0.01
    block.update(0.0, lr)
    for name in ("norm_in", "norm_out", "gate"):
        assert torch.equal(block.params[name], before[name])
    parts = [(n, i, sl) for n, sl in (("down", slice(None)), ("gate_up", slice(0, I)), ("gate_up", slice(I, None)))
             for i in range(cfg["num_experts"])]
    for name, i, sl in parts:
        g = block.grads[name][i, sl]
        scale = -lr * max(1.0, g.shape[0] / g.shape[1]) ** 0.5
        ref, bound = ref_orthogonalize(g, 5, (3.4445, -4.7750, 2.0315), 1e-7, scale, BF)
        step = block.params[name][i, sl].double() - before[name][i, sl].double()
        rounded = 2.0 ** -8 * torch.linalg.vector_norm(block.params[name][i, sl].double())  # the weights' own
        assert float(torch.linalg.vector_norm(step - ref)) <= bound + float(rounded), (name, i)


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_of_one_token_through_layer_norms(captured):
    """Norm, layer, residual sum and norm of what comes next, each on what the one
    before left, against the definitions in 64 bits on the same inputs."""
    T, H, I, E, k = 3, 264, 136, 6, 2
    gen = torch.Generator("cuda").manual_seed(0)
    rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(BF)
    x, ln1, lb1, ln2 = rand(T, H), rand(H), rand(H), rand(H)
    wg, wu, wd, wr = rand(E, I, H, scale=H ** -0.5), rand(E, I, H, scale=H ** -0.5), rand(E, H, I, scale=I ** -0.5), rand(E, H, scale=H ** -0.5)
    h, out, s, n = (torch.empty(T, H, device="cuda", dtype=BF) for _ in range(4))
    logits, w, idx = torch.empty(T, E, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    work = torch.empty(sm.moe_few_tokens_workspace(T, I, k), dtype=torch.uint8, device="cuda")

    def step():
        sm.moe_layer_norm(x, h, w=ln1, b=lb1)
        sm.moe_few_tokens(h, wg, wu, wd, logits, idx, w, out, work, w_router=wr)
        sm.moe_layer_norm(x, n, w=ln2, add=out, sum=s)

    if captured:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
            with torch.cuda.graph(graph, stream=side):
                step()
        torch.cuda.current_stream().wait_stream(side)
        for t in (h, out, s, n, logits, w, idx):
            t.zero_()
        graph.replay()
    else:
        step()
    torch.cuda.synchronize()
    ref, mag = ref_layer_norm(x, ln1, lb1, None, 1e-5)["h"]
    assert bool(((h.double() - ref).abs() <= UNIT[BF] * ref.abs() + 1e-5 * mag * 1.01).all())
    want, weights = ref_route(logits, k)
    assert idx.tolist() == want
    ref, bound = ref_few_tokens(h, wg, wu, wd, want, weights, [[False] * k] * T)
    assert bool(((out.double() - ref).abs() <= bound).all())
    for name, got in (("sum", s), ("h", n)):
        ref, mag = ref_layer_norm(x, ln2, None, out, 1e-5)[name]
        assert bool(((got.double() - ref).abs() <= UNIT[BF] * ref.abs() + 1e-5 * mag * 1.01).all()), name


@pytest.mark.parametrize("update", ["plain", "orthogonal"])
def test_example_runs(update, monkeypatch):
    ex = example()
    monkeypatch.setattr("sys.argv", ["train_moe_block.py", "--steps", "3", "--tokens-per-slot", "16", "--update", update])
    first, last = ex.main()
    assert first == first and last == last  # numbers


def test_calls_on_two_streams_at_once():
    """Two layers and two updates on streams of their own, workspaces apart, give what each gives alone."""
    gen = torch.Generator("cuda").manual_seed(1)
    rand = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(BF)
    jobs = []
    for T, H, I, E, k in ((4, 520, 264, 8, 2), (9, 264, 520, 5, 3)):
        x, wg, wu, wd, lg = rand(T, H), rand(E, I, H, scale=H ** -0.5), rand(E, I, H, scale=H ** -0.5), rand(E, H, I, scale=I ** -0.5), torch.randn(T, E, generator=gen, device="cuda")
        out, w, idx = torch.empty_like(x), torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
        work = torch.empty(sm.moe_few_tokens_workspace(T, I, k), dtype=torch.uint8, device="cuda")
        jobs.append((lambda s, a=(x, wg, wu, wd, lg, idx, w, out, work): sm.moe_few_tokens(*a, stream=s), out))
    for shape in ((2, 300, 200), (1, 129, 600)):
        g = rand(*shape)
        out, work = torch.empty_like(g), torch.empty(sm.moe_orthogonalize_workspace(*shape), dtype=torch.uint8, device="cuda")
        jobs.append((lambda s, a=(g, out, work): sm.moe_orthogonalize(*a, stream=s), out))
    alone = []
    for job, out in jobs:
        job(None)
        torch.cuda.synchronize()
        alone.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        for (job, _), s in zip(jobs, streams):
            job(s)
    torch.cuda.synchronize()
    for (_, out), want in zip(jobs, alone):
        assert torch.equal(out, want)
