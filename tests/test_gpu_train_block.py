"""One training step of an MoE block, made of the library's calls, against the
same block in torch autograd (64 bits) on the library's routing."""
import os
import sys

import pytest
import torch

import moe_synth as ms
from _block_ref import kept

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_moe_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def reference(block, x, dy):
    """(y, gradients) of the block by autograd in 64 bits, routing indices given."""
    cfg, I = block.cfg, block.cfg["inter"]
    p = {k: v.double().requires_grad_() for k, v in block.params.items()}
    x = x.double().requires_grad_()
    norm = lambda t, w: t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    h = norm(x, p["norm_in"])
    idx = block.idx.long()
    w = torch.softmax((h @ p["router"].T).gather(1, idx), 1)
    out = torch.zeros_like(h)
    for e in range(cfg["num_experts"]):
        token, j = (idx == e).nonzero(as_tuple=True)
        gu = h[token] @ p["gate_up"][e].T
        g, u = gu[:, :I], gu[:, I:]
        rows = (w[token, j, None] * torch.nn.functional.silu(g) * u) @ p["down"][e].T
        out = out.index_add(0, token, rows)
    b = torch.tanh(p["gate"]) * norm(out, p["norm_out"])
    b = torch.where(kept(block.seed, block.step, b.shape, block.p), b / (1 - block.p), torch.zeros_like(b))
    y = x + block.scale * b
    y.backward(dy.double())
    return y.detach(), {**{k: v.grad for k, v in p.items()}, "x": x.grad}


@pytest.mark.parametrize("cfg", [ms.shape_of(ms.CONFIGS["tiny"]),
                                 dict(world=2, tokens_per_slot=200, hidden=256, num_experts=8, topk=3, inter=384)])
def test_step_against_autograd(cfg):
    dev = torch.device("cuda")
    block = ex.MoeBlock(cfg, device=dev)
    gen = torch.Generator("cuda").manual_seed(3)
    for t in (block.params["norm_in"], block.params["norm_out"], block.params["gate"]):
        t += (0.2 * torch.randn(t.shape, generator=gen, device=dev)).bfloat16()
    block.params["router"] *= 8  # routing weights away from uniform
    x = ms.x_torch(cfg, dev)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dy = torch.randn(x.shape, generator=gen, device=dev).bfloat16()
    block.forward(x, y)
    block.backward(dy, dx)
    assert block.heap.status() == 0 and block.grad_heap.status() == 0
    ry, rg = reference(block, x, dy)
    # a result passes through at most about ten tensors rounded to 8 bits (half a
    # unit: 2^-9 of the norm each, independent): 2^-9 * sqrt(10) = 0.6 %; the
    # bound takes them as all of one sign, 2 %
    assert float((y.double() - ry).norm() / ry.norm()) < 0.02
    got = {**block.grads, "x": dx}
    for name, ref in rg.items():
        rel = float((got[name].double() - ref).norm() / ref.norm())
        assert rel < 0.02, (name, rel)


def test_example_trains():
    argv, sys.argv = sys.argv, ["train_moe_block.py", "--steps", "12"]
    try:
        first, last = ex.main()
    finally:
        sys.argv = argv
    assert last < first
