"""Host-side checks (no GPU) of the calls for layer norm, orthogonalised updates
and the MoE layer for a few tokens: their structs match the header, and bad
arguments are refused before any device work."""
import ctypes
import os
import subprocess

import pytest
import torch

import combine_symmetric_heap_gb300 as sm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 41  # an aligned address that is never dereferenced on these paths
B = A + (1 << 30)


@pytest.mark.parametrize("name,cls", [("sym_layer_norm", sm.SymLayerNorm), ("sym_layer_norm_grad", sm.SymLayerNormGrad),
                                      ("sym_orthogonalize", sm.SymOrthogonalize), ("sym_few_tokens", sm.SymFewTokens)])
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


def norm(**kw):
    a = dict(rows=4, cols=64, dtype=sm.SYM_BF16, x=A, h=B, ld_x=64, ld_add=64, ld_sum=64, ld_h=64, eps=1e-5)
    a.update(kw)
    return sm.lib().moe_layer_norm(ctypes.byref(sm.SymLayerNorm(**a)), 0)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 30), dict(cols=0), dict(cols=65537), dict(dtype=3), dict(dtype=-1), dict(x=0), dict(x=A + 1),
    dict(h=B + 1), dict(h=0), dict(add=A + 1), dict(sum=B + 1), dict(w=A + 1), dict(b=A + 1), dict(mean=A + 2), dict(rstd=A + 2),
    dict(ld_x=63), dict(ld_h=63), dict(add=A, ld_add=63), dict(sum=A, ld_sum=63), dict(sum=B), dict(eps=-1.0),
    dict(eps=float("nan")), dict(ld_x=1 << 31), dict(dtype=sm.SYM_FP32, x=A + 2),
])
def test_layer_norm_refuses(kw):
    assert norm(**kw) == sm.SYM_EINVAL


def norm_bwd(**kw):
    a = dict(rows=4, cols=64, dtype=sm.SYM_BF16, dh=A, s=A, mean=A, rstd=A, dx=B, ld_dh=64, ld_s=64, ld_dsum=64, ld_dx=64)
    a.update(kw)
    return sm.lib().moe_layer_norm_bwd(ctypes.byref(sm.SymLayerNormGrad(**a)), 0)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=1 << 30), dict(cols=0), dict(cols=65537), dict(dtype=3), dict(dh=0), dict(s=0), dict(mean=0),
    dict(rstd=0), dict(dx=0), dict(dh=A + 1), dict(s=A + 1), dict(dsum=A + 1), dict(w=A + 1), dict(dx=B + 1), dict(dw=B + 1),
    dict(db=B + 1), dict(mean=A + 2), dict(rstd=A + 1), dict(ld_dh=63), dict(ld_s=63), dict(ld_dx=63), dict(dsum=A, ld_dsum=63),
    dict(work=A + 8),
])
def test_layer_norm_bwd_refuses(kw):
    assert norm_bwd(**kw) == sm.SYM_EINVAL


def test_layer_norm_of_no_rows_is_not_an_error():
    assert norm(rows=0, x=0, h=0) == sm.SYM_OK
    assert norm_bwd(rows=0, dh=0, s=0, mean=0, rstd=0) == sm.SYM_OK


def orth(**kw):
    a = dict(count=2, rows=16, cols=32, steps=5, g_dtype=sm.SYM_BF16, out_dtype=sm.SYM_BF16, coeffs=(ctypes.c_float * 3)(3, -4, 2),
             eps=1e-7, scale=1.0, g=A, out=B, g_stride=512, ld_g=32, out_stride=512, ld_out=32, work=A, work_bytes=1 << 40)
    a.update(kw)
    return sm.lib().moe_orthogonalize(ctypes.byref(sm.SymOrthogonalize(**a)), 0)


@pytest.mark.parametrize("kw", [
    dict(count=-1), dict(count=65536), dict(rows=0), dict(rows=65537), dict(cols=0), dict(cols=65537), dict(steps=-1),
    dict(steps=65), dict(g_dtype=3), dict(out_dtype=sm.SYM_FP32), dict(out_dtype=-1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(g=0), dict(out=0), dict(g=A + 1), dict(out=B + 1), dict(g_dtype=sm.SYM_FP32, g=A + 2), dict(ld_g=31), dict(ld_out=31),
    dict(g_stride=511), dict(out_stride=511), dict(work=A + 128),
])
def test_orthogonalize_refuses(kw):
    assert orth(**kw) == sm.SYM_EINVAL


def test_orthogonalize_of_nothing_is_not_an_error():
    assert orth(count=0, g=0, out=0, work=0, work_bytes=0) == sm.SYM_OK


def few(**kw):
    a = dict(tokens=4, hidden=64, inter=128, num_experts=8, topk=2, dtype=sm.SYM_BF16, x=A, w_gate=A, w_up=A, w_down=A, logits=A,
             idx=A, w=A, out=B, ld_x=64, ld_out=64, gate_group=64 * 128, gate_ld=64, up_group=64 * 128, up_ld=64,
             down_group=64 * 128, down_ld=128, router_ld=64, work=A, work_bytes=1 << 40)
    a.update(kw)
    return sm.lib().moe_few_tokens(ctypes.byref(sm.SymFewTokens(**a)), 0)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=33), dict(hidden=0), dict(hidden=60), dict(hidden=65544), dict(inter=0), dict(inter=124),
    dict(inter=65544), dict(num_experts=0), dict(num_experts=1025), dict(num_experts=1), dict(topk=0), dict(topk=9),
    dict(topk=33, num_experts=64), dict(dtype=sm.SYM_FP32), dict(dtype=-1), dict(x=0), dict(x=A + 8), dict(w_gate=0),
    dict(w_gate=A + 8), dict(w_up=0), dict(w_up=A + 2), dict(w_down=0), dict(w_down=A + 4), dict(w_router=A + 8),
    dict(logits=0), dict(logits=A + 2), dict(idx=0), dict(idx=A + 1), dict(w=0), dict(w=A + 2), dict(out=0), dict(out=B + 1),
    dict(ld_x=68), dict(ld_x=56), dict(ld_out=63), dict(gate_ld=56), dict(gate_ld=68), dict(up_ld=56), dict(down_ld=120),
    dict(down_ld=132), dict(gate_group=64), dict(up_group=64 * 128 + 4), dict(down_group=64 * 127), dict(w_router=A, router_ld=56),
    dict(work=A + 8),
])
def test_few_tokens_refuses(kw):
    assert few(**kw) == sm.SYM_EINVAL


def test_few_tokens_of_none_is_not_an_error():
    assert few(tokens=0, x=0, logits=0, idx=0, w=0, out=0, work=0, work_bytes=0) == sm.SYM_OK


def test_few_tokens_workspace():
    n = sm.moe_few_tokens_workspace(4, 128, 2)
    assert n >= 4 * 2 * 128 * 4
    for bad in ((33, 128, 2), (-1, 128, 2), (4, 124, 2), (4, 0, 2), (4, 128, 0), (4, 128, 33)):
        with pytest.raises(sm.SymmoeError) as e:
            sm.moe_few_tokens_workspace(*bad)
        assert e.value.code == sm.SYM_EINVAL


def test_tensors_off_the_device_are_refused():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    calls = [lambda: sm.moe_layer_norm(x, x),
             lambda: sm.moe_layer_norm_bwd(x, x, x, x, dx=x),
             lambda: sm.moe_orthogonalize(x, x, x),
             lambda: sm.moe_few_tokens(x, x, x, x, x, x, x, x, x)]
    for call in calls:
        with pytest.raises(sm.SymmoeError) as e:
            call()
        assert e.value.code == sm.SYM_EINVAL
