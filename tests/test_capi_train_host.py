"""Host-side checks (no GPU) of the calls for training through an MoE block:
their structs match the header, and bad arguments are refused before any device
work."""
import ctypes
import os
import subprocess

import pytest
import torch

import combine_symmetric_heap_gb300 as sm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 41  # an aligned address that is never dereferenced on these paths
NO = None


@pytest.mark.parametrize("name,cls", [("sym_rows", sm.SymRows), ("sym_groups", sm.SymGroups),
                                      ("sym_block_norm", sm.SymBlockNorm), ("sym_block_norm_grad", sm.SymBlockNormGrad)])
def test_struct_layout_matches_header(tmp_path, name, cls):
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    lines = ["#include <stdio.h>", "#include <stddef.h>", f'#include "{os.path.join(ROOT, "include", "symmoe.h")}"',
             "int main(void){", f'printf("size %zu\\n", sizeof({name}));']
    lines += [f'printf("{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_] + ["return 0;}"]
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-o", str(exe), str(src)], check=True)
    out = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(cls)
    for f in cls._fields_:
        assert int(out[f[0]]) == getattr(cls, f[0]).offset, f[0]


def rows(n=16, cols=64, ld=None, slots=1, stride=0, ptr=A):
    return sm.SymRows(ptr, ld or cols, stride, n, slots, cols)


def groups(n=2, slots=1, cnt=A, off=A, stride=0):
    return sm.SymGroups(cnt, off, stride, stride, 0, n, slots, 0, 0)


def matmul(g=NO, dtype=0, x=NO, w=A, ws=4096, wl=64, flags=0, out=NO):
    r = ctypes.byref
    return sm.lib().moe_grouped_matmul(r(g or groups()), dtype, r(x or rows()), w, ws, wl, flags, r(out or rows()), 0)


def wgrad(g=NO, dtype=0, dy=NO, x=NO, dw=A, ws=4096, wl=64, odt=0, flags=0):
    r = ctypes.byref
    return sm.lib().moe_grouped_wgrad(r(g or groups()), dtype, r(dy or rows()), r(x or rows()), dw, ws, wl, odt, flags, 0)


@pytest.mark.parametrize("kw", [
    dict(dtype=sm.SYM_FP32), dict(dtype=7), dict(flags=2), dict(w=NO), dict(w=A + 8), dict(wl=60), dict(wl=32),
    dict(ws=64), dict(ws=4100), dict(x=rows(ptr=A + 2)), dict(x=rows(ld=68)), dict(x=rows(ld=32)), dict(x=rows(cols=0)),
    dict(x=rows(cols=65537, ld=65600)), dict(x=rows(n=-1)), dict(x=rows(n=1 << 30)), dict(out=rows(n=15)),
    dict(out=rows(ptr=A + 1)), dict(out=rows(slots=2, stride=4096)), dict(g=groups(n=0)), dict(g=groups(n=1025)),
    dict(g=groups(cnt=0)), dict(g=groups(off=A + 2)), dict(g=groups(n=2, slots=2)),
    dict(g=groups(n=3, slots=2, stride=2), x=rows(slots=2, stride=1024), out=rows(slots=2, stride=1024)),
    dict(g=groups(n=4, slots=2, stride=1), x=rows(slots=2, stride=1024), out=rows(slots=2, stride=1024)),
    dict(g=groups(n=4, slots=2, stride=2), x=rows(slots=2, stride=1020), out=rows(slots=2, stride=1024)),
])
def test_grouped_matmul_refuses(kw):
    assert matmul(**kw) == sm.SYM_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dtype=sm.SYM_FP32, odt=sm.SYM_FP32), dict(odt=sm.SYM_FP16), dict(flags=2), dict(dw=NO), dict(dw=A + 1),
    dict(odt=sm.SYM_FP32, dw=A + 2), dict(wl=32), dict(ws=64), dict(dy=rows(n=15)), dict(dy=rows(ld=68)),
    dict(x=rows(ptr=A + 8)), dict(g=groups(n=2, slots=2)),
])
def test_grouped_wgrad_refuses(kw):
    assert wgrad(**kw) == sm.SYM_EINVAL


def test_nothing_to_do_is_not_an_error():
    assert matmul(x=rows(n=0, ptr=0), out=rows(n=0, ptr=0)) == sm.SYM_OK
    r = ctypes.byref
    e = rows(n=0, ptr=0)
    L = sm.lib()
    assert L.moe_swiglu_rows(2, r(e), r(e), None, 0, None, 0, r(e), 0) == sm.SYM_OK
    assert L.moe_dropout(2, r(e), None, r(e), 0.5, 1, 2, 0) == sm.SYM_OK
    assert L.moe_block_norm(r(sm.SymBlockNorm(rows=0, cols=64, dtype=2)), 0) == sm.SYM_OK
    out = ctypes.c_uint64()
    bad = [(-1, 64, 0), (4, 0, 0), (4, 65537, 0), (4, 64, 3), (4, 64, 5), (1 << 30, 64, 0)]
    assert all(L.moe_block_norm_workspace(*a, r(out)) == sm.SYM_EINVAL for a in bad)


def test_row_calls_refuse():
    r, L = ctypes.byref, sm.lib()
    x, odd, few = rows(), rows(ptr=A + 2), rows(n=15)
    for bad in ((3, x, x, x), (2, odd, x, x), (2, x, few, x), (2, x, x, rows(cols=63)), (2, x, x, rows(ptr=0))):
        assert L.moe_swiglu_rows(bad[0], r(bad[1]), r(bad[2]), None, 0, None, 0, r(bad[3]), 0) == sm.SYM_EINVAL
    assert L.moe_swiglu_rows(2, r(x), r(x), A + 2, 0, None, 0, r(x), 0) == sm.SYM_EINVAL
    assert L.moe_swiglu_rows(2, r(x), r(x), None, 0, A + 1, 0, r(x), 0) == sm.SYM_EINVAL
    assert L.moe_swiglu_rows_bwd(2, r(x), r(x), r(x), None, 0, None, 0, r(x), r(few), None, 0, 0) == sm.SYM_EINVAL
    assert L.moe_swiglu_rows_bwd(2, r(x), r(x), r(x), None, 0, None, 0, r(x), r(x), A + 2, 0, 0) == sm.SYM_EINVAL
    for p in (1.0, -0.1, float("nan"), float("inf")):
        assert L.moe_dropout(2, r(x), None, r(x), p, 0, 0, 0) == sm.SYM_EINVAL
    assert L.moe_dropout(2, r(x), r(few), r(x), 0.1, 0, 0, 0) == sm.SYM_EINVAL


def block(**kw):
    base = dict(rows=4, cols=64, dtype=2, x=A, o=A, y=A, h=A, ld_x=64, ld_o=64, ld_y=64, ld_h=64, scale=1.0)
    return sm.SymBlockNorm(**{**base, **kw})


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(rows=-1), dict(rows=1 << 30), dict(cols=0), dict(cols=65537), dict(flags=2), dict(gate_act=3),
    dict(p=1.0), dict(p=float("nan")), dict(eps=-1.0), dict(x=0), dict(y=0), dict(o=0), dict(o=0, y=0, h=0), dict(x=A + 2),
    dict(ld_x=63), dict(ld_h=1 << 31), dict(gate=A, ld_gate=64), dict(gate=A, ld_gate=64, gate_rows=3),
    dict(gate=A, ld_gate=64, gate_rows=8), dict(gate=A, ld_gate=32, gate_rows=2), dict(w_post=A, flags=1),
    dict(rstd_post=A, flags=1), dict(rstd_pre=A + 2), dict(o=0, y=0, gate=A, gate_rows=1, ld_gate=64),
])
def test_block_norm_refuses(kw):
    assert sm.lib().moe_block_norm(ctypes.byref(block(**kw)), 0) == sm.SYM_EINVAL


@pytest.mark.parametrize("kw,grad", [
    (dict(), dict()), (dict(), dict(dy=A, ld_dy=63)), (dict(), dict(dh=A, ld_dh=64)), (dict(), dict(dy=A, ld_dy=64)),
    (dict(o=0), dict(dy=A, ld_dy=64, d_o=A, ld_do=64)), (dict(rstd_post=A), dict(dy=A, ld_dy=64, dgate=A, ld_dgate=64)),
    (dict(rstd_post=A), dict(dy=A, ld_dy=64, dw_pre=A)), (dict(flags=1), dict(dy=A, ld_dy=64, dw_post=A)),
    (dict(rstd_post=A), dict(dy=A, ld_dy=64, work=A + 8)),
])
def test_block_norm_bwd_refuses(kw, grad):
    g = sm.SymBlockNormGrad(**grad)
    assert sm.lib().moe_block_norm_bwd(ctypes.byref(block(**kw)), ctypes.byref(g), 0) == sm.SYM_EINVAL


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64)
    n = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: sm.moe_dropout(x, x, 0.1, 0), lambda: sm.moe_swiglu_rows(x, x, x),
                 lambda: sm.moe_block_norm(x, h=x), lambda: sm.moe_block_norm_bwd(dy=x, dx=x),
                 lambda: sm.moe_grouped_matmul(x, x[None], n, n, x), lambda: sm.moe_grouped_wgrad(x, x, n, n, x[None])):
        with pytest.raises(sm.SymmoeError) as ei:
            call()
        assert ei.value.code == sm.SYM_EINVAL
