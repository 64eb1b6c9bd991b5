"""Numbers that the argument structs cannot hold are refused like any other bad argument (no
GPU: the tensors are taken as if the CPU were the current device)."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(sm, "_device", lambda: torch.zeros(1).get_device())


def refused(call):
    with pytest.raises(sm.SymmoeError) as e:
        call()
    assert e.value.code == sm.SYM_EINVAL


@pytest.mark.parametrize("kw", [dict(steps=1 << 40), dict(steps=-(1 << 40)), dict(steps=2.5), dict(steps=None), dict(eps=None),
                                dict(scale="1"), dict(coeffs=(None, 0.0, 0.0)), dict(coeffs=(1.0, "b", 0.0)), dict(wait_timeout_us=-1), dict(wait_timeout_us=1 << 32)])
def test_orthogonalize(kw):
    g = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    refused(lambda: sm.moe_orthogonalize(g, torch.empty_like(g), torch.empty(1 << 20, dtype=torch.uint8), **kw))


@pytest.mark.parametrize("kw", [dict(eps=None), dict(eps="1")])
def test_layer_norm(kw):
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    refused(lambda: sm.moe_layer_norm(x, torch.empty_like(x), **kw))


def test_sizes_beyond_32_bits():
    g = torch.empty(0, 8, 1 << 31, dtype=torch.bfloat16)
    refused(lambda: sm.moe_orthogonalize(g, g, torch.empty(0, dtype=torch.uint8)))
    refused(lambda: sm.moe_layer_norm(torch.empty(0, 1 << 31, dtype=torch.bfloat16), torch.empty(0, 1 << 31, dtype=torch.bfloat16)))
