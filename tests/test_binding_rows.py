"""Host-side checks (no GPU) of what the binding reads from tensors' shapes and
strides for the training calls."""
import pytest
import torch

import combine_symmetric_heap_gb300 as sm


def refused(call, *a):
    with pytest.raises(sm.SymmoeError) as ei:
        call(*a)
    assert ei.value.code == sm.SYM_EINVAL


def test_totals_are_one_word_for_each_slot():
    """The slot stride that is read from `total` stays inside the tensor."""
    rows = sm._rows(torch.zeros(3, 4, 8), "t")
    words = torch.arange(6, dtype=torch.int32)
    for t in (words[:3], words[::2], words[:3].view(3, 1), words.view(3, 2)[:, :1], words[:1].expand(3)):
        ptr, stride = sm._totals(t, rows, "t")
        room = t.untyped_storage().nbytes() // 4
        assert ptr == t.data_ptr() and [t.storage_offset() + d * stride for d in range(3)] == \
            [t.storage_offset() + d * t.stride(0) for d in range(3)] and t.storage_offset() + 2 * stride < room
    for bad in (words[:3].view(1, 3), words.view(2, 3)[:, :1], words[:2], words[:3].long(), words[:3].view(3, 1, 1)):
        refused(sm._totals, bad, rows, "t")
    one = sm._rows(torch.zeros(4, 8), "t")
    for t in (words[1], words[1:2], words[1:2].view(1, 1)):
        assert sm._totals(t, one, "t") == (t.data_ptr(), 0)
    refused(sm._totals, words[:2], one, "t")


def test_no_slots():
    words = torch.zeros(2, dtype=torch.int32)
    refused(sm._groups, words, words, sm._rows(torch.zeros(0, 4, 8), "t"), None, "t")


def norm_args(rows, gate):
    x = torch.zeros(rows, 8)
    return ("t", x.dtype, rows, 8, x, x, None, gate, "none", 1.0, 0.0, 0, 0, None, x, None, None, None, True, 1e-6)


def test_gate_without_rows():
    """An empty gate is no gate row for rows that are there (and not the absence of a gate)."""
    refused(sm._block, *norm_args(4, torch.zeros(0, 8)))
    assert sm._block(*norm_args(0, torch.zeros(0, 8))).gate_rows == 0
    assert sm._block(*norm_args(4, torch.zeros(2, 8))).gate_rows == 2
