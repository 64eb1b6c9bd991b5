"""A wait of the orthogonalised updates that runs out reaches the caller."""
import importlib.util
import inspect
import os

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
import moe_synth as ms

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_binding_takes_a_wait_limit():
    """Waits limited to 20 us where a tile's K axis takes about a millisecond; the call after it is whole again."""
    rows, cols = 600, 65536
    g = torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(0), device="cuda").half()
    out, status = torch.empty_like(g), torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.empty(sm.moe_orthogonalize_workspace(1, rows, cols), dtype=torch.uint8, device="cuda")
    sm.moe_orthogonalize(g, out, work, steps=1, status=status, wait_timeout_us=1000000)
    want = out.clone()
    assert int(status) == 0
    sm.moe_orthogonalize(g, out, work, steps=1, status=status, wait_timeout_us=20)
    assert int(status) & sm.SYM_STATUS_TIMEOUT
    status.zero_()
    sm.moe_orthogonalize(g, out, work, steps=1, status=status)
    assert int(status) == 0 and torch.equal(out, want)


def test_the_example_looks_for_it(monkeypatch):
    """Every update of the example has the heap's status word, which its step checks."""
    spec = importlib.util.spec_from_file_location("train_moe_block", os.path.join(ROOT, "examples", "train_moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    real, seen = sm.moe_orthogonalize, []

    def spy(*a, **kw):
        seen.append(inspect.signature(real).bind(*a, **kw).arguments.get("status"))
        real(*a, **kw)

    monkeypatch.setattr(sm, "moe_orthogonalize", spy)
    block = ex.MoeBlock(dict(ms.shape_of(ms.CONFIGS["tiny"]), tokens_per_slot=16), dropout=0.0)
    x = ms.x_torch(block.cfg, torch.device("cuda"))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    block.forward(x, y)
    block.backward(x, dx)
    block.update(0.0, 0.01)
    assert len(seen) == 4 and all(s is not None and s.data_ptr() == block.heap.status_word().data_ptr() for s in seen)
    monkeypatch.setattr(sm, "moe_orthogonalize", lambda *a, **kw: kw["status"].fill_(sm.SYM_STATUS_TIMEOUT))
    monkeypatch.setattr("sys.argv", ["train_moe_block.py", "--steps", "1", "--tokens-per-slot", "16", "--update", "orthogonal"])
    with pytest.raises(AssertionError):
        ex.main()
