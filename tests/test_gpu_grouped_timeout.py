"""Grouped products whose internal waits run out: the status word says so, the
launch ends, and the device goes on working."""
import ctypes

import pytest
import torch

import combine_symmetric_heap_gb300 as sm
from _block_ref import assert_within, groups_of, product_bound, ref_product, ref_wgrad

pytestmark = pytest.mark.gpu


def groups(cnt, off, status, limit_us):
    return sm.SymGroups(cnt.data_ptr(), off.data_ptr(), 0, 0, status.data_ptr(), cnt.numel(), 1, limit_us, 0)


def rows(t):
    return sm._rows(t, "t")


def wgrad(dy, x, dw, g):
    r = ctypes.byref
    return sm.lib().moe_grouped_wgrad(r(g), sm.SYM_BF16, r(rows(dy)), r(rows(x)), dw.data_ptr(), dw.stride(0), dw.stride(1),
                                      sm.SYM_BF16, 0, None)


def matmul(x, w, out, g, flags):
    r = ctypes.byref
    return sm.lib().moe_grouped_matmul(r(g), sm.SYM_BF16, r(rows(x)), w.data_ptr(), w.stride(0), w.stride(1), flags,
                                       r(rows(out)), None)


def small_calls_are_right():
    gen = torch.Generator(device="cuda").manual_seed(1)
    cnt, off, n = groups_of([300, 0, 77])
    x = torch.randn(1, n, 136, generator=gen, device="cuda").bfloat16()
    w = torch.randn(3, 264, 136, generator=gen, device="cuda").bfloat16()
    out, dw = torch.empty(1, n, 264, device="cuda", dtype=torch.bfloat16), torch.empty_like(w)
    sm.moe_grouped_matmul(x, w, cnt, off, out)
    sm.moe_grouped_wgrad(out, x, cnt, off, dw)
    ref, mag, _ = ref_product(x, w, cnt, off, False)
    assert_within(out, ref, mag, "product", product_bound(136))
    ref, mag = ref_wgrad(out, x, cnt, off)
    assert_within(dw, ref, mag, "wgrad", product_bound(300))


def test_weight_gradient_whose_waits_run_out():
    """One tile of 2^20 - 3 rows, some milliseconds of contraction, under a limit of
    20 us (and with rows for the side buffer)."""
    n = (1 << 20) - 3
    x = torch.zeros(n, 64, device="cuda", dtype=torch.bfloat16)
    dw = torch.zeros(1, 64, 64, device="cuda", dtype=torch.bfloat16)
    cnt, off = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert wgrad(x, x, dw, groups(cnt, off, status, 20)) == sm.SYM_OK
    torch.cuda.synchronize()
    assert int(status) == sm.SYM_STATUS_TIMEOUT
    small_calls_are_right()
    status.zero_()  # under the default limit the same call has time
    assert wgrad(x, x, dw, groups(cnt, off, status, 0)) == sm.SYM_OK
    torch.cuda.synchronize()
    assert int(status) == 0


@pytest.mark.parametrize("flags", [0, sm.SYM_GM_TRANS_W])
def test_product_under_a_short_limit(flags):
    """The longest contraction is some hundred microseconds: the waits may or may not
    run out under the shortest limit; the call ends either way, and says which."""
    C, F, n = 65536, 512, 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n, C, generator=gen, device="cuda").bfloat16()
    w = torch.randn((1, C, F) if flags else (1, F, C), generator=gen, device="cuda").bfloat16()
    out, want = (torch.empty(n, F, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cnt, off = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert matmul(x, w, out, groups(cnt, off, status, 1), flags) == sm.SYM_OK
    torch.cuda.synchronize()
    assert int(status) in (0, sm.SYM_STATUS_TIMEOUT)
    sm.moe_grouped_matmul(x, w, cnt, off, want, trans_w=bool(flags))
    assert int(status) != 0 or torch.equal(out, want)
    small_calls_are_right()


def test_weight_gradient_that_outlasts_the_limit_of_one_wait():
    """The limit is for a wait, not for the launch: a long group without a remainder
    between short ones with one takes several times the limit, each of its tiles a
    fraction of it."""
    big, C = 200_000, 8192  # about 14 tiles of a millisecond for each pair
    gen = torch.Generator(device="cuda").manual_seed(3)
    cnt, off, n = groups_of([3, big, 5])
    x, dy = (torch.randn(1, n, C, generator=gen, device="cuda", dtype=torch.bfloat16)[0] for _ in range(2))
    dw = torch.empty(3, C, C, device="cuda", dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    assert wgrad(dy, x, dw, groups(cnt, off, status, 4000)) == sm.SYM_OK
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 8, "not the long launch that this is about"
    assert int(status) == 0
    for e, (at, rows_) in enumerate(((0, 3), (3 + big, 5))):
        g = [0, 2][e]
        ref = dy[at:at + rows_].double().T @ x[at:at + rows_].double()
        mag = dy[at:at + rows_].double().abs().T @ x[at:at + rows_].double().abs()
        assert_within(dw[g], ref, mag, "wgrad", product_bound(rows_))
