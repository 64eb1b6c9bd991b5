"""The example's orthogonal update: each matrix, the router's included, takes exactly what the
call gives for its gradient."""
import importlib.util
import os

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
import moe_synth as ms

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [16, 64])
def test_every_matrix_takes_the_update_of_its_gradient(tokens):
    spec = importlib.util.spec_from_file_location("train_moe_block", os.path.join(ROOT, "examples", "train_moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.MoeBlock(dict(ms.shape_of(ms.CONFIGS["tiny"]), tokens_per_slot=tokens), dropout=0.0)
    x = ms.x_torch(block.cfg, torch.device("cuda"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    block.forward(x, y)
    block.backward(x, dx)
    before, I, lr = {n: t.clone() for n, t in block.params.items()}, block.cfg["inter"], 0.01
    block.update(0.0, lr)
    parts = [("router", slice(None), False), ("down", slice(None), True), ("gate_up", slice(0, I), True), ("gate_up", slice(I, None), True)]
    for name, rows, experts in parts:
        at = (slice(None), rows) if experts else (rows,)
        g = block.grads[name][at].contiguous()
        count, (f, c) = g.shape[0] if experts else 1, g.shape[-2:]
        way = torch.empty_like(g)
        sm.moe_orthogonalize(g, way, torch.empty(sm.moe_orthogonalize_workspace(count, f, c), dtype=torch.uint8, device="cuda"),
                             scale=-lr * max(1.0, f / c) ** 0.5)
        assert bool(way.any())
        assert torch.equal(block.params[name][at], before[name][at] + way), name
    for name in ("norm_in", "norm_out", "gate"):
        assert torch.equal(block.params[name], before[name])
