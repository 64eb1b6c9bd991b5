"""Zero-copy MoE dispatch -> expert -> combine over a flat symmetric heap, GB300.

Thin Python binding of the C-ABI library ``libsymmoe.so`` (declared in
``include/symmoe.h``).  Functions keep the C names and only marshal
arguments: torch tensors or raw device addresses in, ``SymmoeError`` on a
non-zero return.  Every step of the path runs in the library's CUDA kernels;
torch is used for device memory and streams only.  There is no CPU fallback:
importing the package fails loudly if the library has not been built
(``python combine_symmetric_heap_gb300/build.py``).

``SymHeap`` is a convenience owner of one heap allocation (a torch uint8
tensor) with zero-copy tensor views of its windows, e.g.
``heap.combine_in_view()`` -- the expert-output window whose ``data_ptr``
``moe_combine`` recognises (MORI CCO blog, "Zero-copy MoE dispatch -> expert
-> combine": combine skips its staging copy when the expert wrote into the
view it handed out).
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libsymmoe.so")

SYM_OK = 0
SYM_EINVAL = -1
SYM_ENOSPACE = -2
SYM_ECUDA = -3
SYM_ETIMEOUT = -4
SYM_EOVERFLOW = -5
SYM_ENOTSUP = -6
SYM_STATUS_TIMEOUT = 0x1
SYM_STATUS_OVERFLOW = 0x2
SYM_ROWS_PER_FLAG = 128
SYM_COUNT_CHUNK = 128
SYM_GUARD_BYTES = 1024
SYM_HEAP_WINDOWS = 13

_u64 = ctypes.c_uint64
_u32 = ctypes.c_uint32
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


class MoeShape(ctypes.Structure):
    _fields_ = [("world", _i32), ("tokens_per_slot", _i32), ("hidden", _i32),
                ("inter", _i32), ("num_experts", _i32), ("topk", _i32)]


class SymHeapDesc(ctypes.Structure):
    _fields_ = [("base", _u64), ("per_rank_size", _u64), ("bytes", _u64), ("cap", _u64),
                ("off_recv_x", _u64), ("off_y", _u64), ("off_h", _u64),
                ("off_recv_pair", _u64), ("off_recv_w", _u64), ("off_pos", _u64),
                ("off_cnt", _u64), ("off_recv_off", _u64), ("off_total", _u64),
                ("off_status", _u64), ("off_ready", _u64), ("off_hist", _u64),
                ("off_ctrl", _u64), ("num_ready", _u32), ("epoch", _u32),
                ("wait_timeout_us", _u32), ("reserved", _u32), ("s", MoeShape)]


class SymRows(ctypes.Structure):
    _fields_ = [("ptr", _u64), ("ld", _i64), ("slot_stride", _i64), ("rows", _i64), ("slots", _i32),
                ("cols", _i32)]


class SymGroups(ctypes.Structure):
    _fields_ = [("cnt", _u64), ("off", _u64), ("cnt_slot_stride", _i64), ("off_slot_stride", _i64),
                ("status", _u64), ("groups", _i32), ("slots", _i32), ("wait_timeout_us", _u32),
                ("reserved", _u32)]


class SymBlockNorm(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i32), ("dtype", _i32), ("x", _u64), ("o", _u64), ("w_post", _u64),
                ("gate", _u64), ("w_pre", _u64), ("y", _u64), ("h", _u64), ("rstd_post", _u64),
                ("rstd_pre", _u64), ("ld_x", _i64), ("ld_o", _i64), ("ld_gate", _i64), ("ld_y", _i64),
                ("ld_h", _i64), ("gate_rows", _i64), ("gate_act", _i32), ("flags", _i32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("p", ctypes.c_double), ("seed", _u64),
                ("offset", _u64)]


class SymBlockNormGrad(ctypes.Structure):
    _fields_ = [("dy", _u64), ("dh", _u64), ("dx", _u64), ("d_o", _u64), ("dw_pre", _u64), ("dw_post", _u64),
                ("dgate", _u64), ("ld_dy", _i64), ("ld_dh", _i64), ("ld_dx", _i64), ("ld_do", _i64),
                ("ld_dgate", _i64), ("work", _u64), ("work_bytes", _u64)]


class SymmoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {sym_strerror(code)} ({code})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libsymmoe.so not built ({LIB_PATH}); run "
                               "python combine_symmetric_heap_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.sym_heap_bytes.argtypes = [P(MoeShape), _u64, P(_u64), P(_u64)]
        L.sym_heap_init.argtypes = [P(MoeShape), _vp, _u64, _u64, P(SymHeapDesc)]
        L.sym_heap_slot_ptr.argtypes = [P(SymHeapDesc), ctypes.c_int, _u64]
        L.sym_heap_slot_ptr.restype = _vp
        L.sym_heap_windows.argtypes = [P(SymHeapDesc), P(_u64), P(_u64), ctypes.c_int]
        L.moe_route_topk.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp]
        L.moe_router_logits.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp]
        L.moe_router_splits.argtypes = [P(SymHeapDesc), P(ctypes.c_int)]
        L.moe_dispatch.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp]
        L.moe_dispatch_ex.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, ctypes.c_int, _vp]
        L.moe_expert_ffn.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp]
        L.moe_expert_ffn_ex.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, ctypes.c_int, _vp]
        L.moe_combine.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp, _vp]
        L.moe_combine_ex.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp, ctypes.c_int, _vp]
        L.moe_combine_fallback_copies.restype = _u64
        L.moe_pipeline.argtypes = [P(SymHeapDesc), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   ctypes.c_int, _vp]
        L.sym_heap_status.argtypes = [P(SymHeapDesc), P(_i32), ctypes.c_int, _vp]
        L.sym_gemm_a2a.argtypes = [P(SymHeapDesc), _vp, _vp, ctypes.c_int, _vp]
        L.sym_a2a_gemm.argtypes = [P(SymHeapDesc), _vp, _vp, ctypes.c_int, _vp]
        L.moe_dispatch_layout_noalloc.argtypes = [P(MoeShape), _vp, _vp, _vp, _vp, _vp, _vp]
        R, G = P(SymRows), P(SymGroups)
        L.moe_grouped_matmul.argtypes = [G, ctypes.c_int, R, _vp, _i64, _i64, ctypes.c_int, R, _vp]
        L.moe_grouped_wgrad.argtypes = [G, ctypes.c_int, R, R, _vp, _i64, _i64, ctypes.c_int, ctypes.c_int, _vp]
        L.moe_swiglu_rows.argtypes = [ctypes.c_int, R, R, _vp, _i64, _vp, _i64, R, _vp]
        L.moe_swiglu_rows_bwd.argtypes = [ctypes.c_int, R, R, R, _vp, _i64, _vp, _i64, R, R, _vp, _i64, _vp]
        L.moe_dropout.argtypes = [ctypes.c_int, R, R, R, ctypes.c_double, _u64, _u64, _vp]
        L.moe_block_norm.argtypes = [P(SymBlockNorm), _vp]
        L.moe_block_norm_bwd.argtypes = [P(SymBlockNorm), P(SymBlockNormGrad), _vp]
        L.moe_block_norm_workspace.argtypes = [_i64, _i32, _i64, P(_u64)]
        L.sym_strerror.argtypes = [ctypes.c_int]
        L.sym_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _stream(s) -> int | None:
    if s is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(s, torch.cuda.Stream):
        return s.cuda_stream
    return int(s)


def _check(rc: int, where: str) -> None:
    if rc != SYM_OK:
        raise SymmoeError(rc, where)


def _shape(shape) -> MoeShape:
    if isinstance(shape, MoeShape):
        return shape
    return MoeShape(shape["world"], shape["tokens_per_slot"], shape["hidden"], shape["inter"],
                    shape["num_experts"], shape["topk"])


# ------------------------------------------------------------------ C calls

def sym_strerror(code: int) -> str:
    return lib().sym_strerror(code).decode()


def sym_heap_bytes(shape, align: int = 0):
    prs, tot = _u64(), _u64()
    s = _shape(shape)
    _check(lib().sym_heap_bytes(ctypes.byref(s), align, ctypes.byref(prs), ctypes.byref(tot)),
           "sym_heap_bytes")
    return prs.value, tot.value


def sym_heap_init(shape, dev_base, nbytes: int, align: int = 0) -> SymHeapDesc:
    out = SymHeapDesc()
    s = _shape(shape)
    _check(lib().sym_heap_init(ctypes.byref(s), _ptr(dev_base), nbytes, align, ctypes.byref(out)),
           "sym_heap_init")
    return out


def sym_heap_slot_ptr(heap: SymHeapDesc, slot: int, offset: int) -> int | None:
    return lib().sym_heap_slot_ptr(ctypes.byref(heap), slot, offset)


def moe_route_topk(heap: SymHeapDesc, logits, idx, w, stream=None) -> None:
    _check(lib().moe_route_topk(ctypes.byref(heap), _ptr(logits), _ptr(idx), _ptr(w),
                                _stream(stream)), "moe_route_topk")


def moe_router_logits(heap: SymHeapDesc, x, w_router, logits, stream=None) -> None:
    _check(lib().moe_router_logits(ctypes.byref(heap), _ptr(x), _ptr(w_router), _ptr(logits),
                                   _stream(stream)), "moe_router_logits")


def moe_router_splits(heap: SymHeapDesc) -> int:
    out = ctypes.c_int(0)
    _check(lib().moe_router_splits(ctypes.byref(heap), ctypes.byref(out)), "moe_router_splits")
    return out.value


def moe_dispatch(heap: SymHeapDesc, x, idx, w, stream=None) -> None:
    _check(lib().moe_dispatch(ctypes.byref(heap), _ptr(x), _ptr(idx), _ptr(w), _stream(stream)),
           "moe_dispatch")


def moe_expert_ffn(heap: SymHeapDesc, w_gate, w_up, w_down, stream=None) -> None:
    _check(lib().moe_expert_ffn(ctypes.byref(heap), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                _stream(stream)), "moe_expert_ffn")


def moe_combine(heap: SymHeapDesc, expert_out, idx, w, out, stream=None) -> None:
    _check(lib().moe_combine(ctypes.byref(heap), _ptr(expert_out), _ptr(idx), _ptr(w), _ptr(out),
                             _stream(stream)), "moe_combine")


# flags of the _ex calls and pipeline modes (include/symmoe.h)
SYM_FFN_WEIGHTED_ROWS = 1
SYM_COMBINE_UNWEIGHTED = 1
SYM_PIPE_FUSED = 1
SYM_PIPE_WEIGHTS_IN_FFN = 2
SYM_PIPE_DEDUP = 4
SYM_PIPE_FP8 = 8
SYM_LA_FUSED = 1
SYM_DISPATCH_DEDUP = 1
SYM_DISPATCH_FP8 = 2
SYM_LA_COPY_ENGINES = 2


def sym_gemm_a2a(heap: SymHeapDesc, x, w, mode: int = 0, stream=None) -> None:
    """GEMM -> all-to-all: slot s's rows of x through w, exchanged in W row
    blocks into the y windows (mode SYM_LA_FUSED: the epilogue stores at the
    destination; 0: GEMM, then a copy kernel)."""
    _check(lib().sym_gemm_a2a(ctypes.byref(heap), _ptr(x), _ptr(w), int(mode), _stream(stream)),
           "sym_gemm_a2a")


def sym_a2a_gemm(heap: SymHeapDesc, z, w, mode: int = 0, stream=None) -> None:
    """All-to-all -> GEMM: K-shards z [W][N][H/W] gathered per slot, then w;
    results in the y windows (mode SYM_LA_FUSED: the GEMM reads each shard in
    place; SYM_LA_FUSED | SYM_LA_COPY_ENGINES: copy-engine copies consumed as
    they land; 0: a copy kernel, then the GEMM)."""
    _check(lib().sym_a2a_gemm(ctypes.byref(heap), _ptr(z), _ptr(w), int(mode), _stream(stream)),
           "sym_a2a_gemm")


def moe_dispatch_ex(heap: SymHeapDesc, x, idx, w, flags: int = 0, stream=None) -> None:
    """flags: SYM_DISPATCH_DEDUP for the rank-deduplicated dispatch (same windows),
    SYM_DISPATCH_FP8 for the FP8 dispatch with per-token scales."""
    _check(lib().moe_dispatch_ex(ctypes.byref(heap), _ptr(x), _ptr(idx), _ptr(w), int(flags),
                                 _stream(stream)), "moe_dispatch_ex")


def moe_expert_ffn_ex(heap: SymHeapDesc, w_gate, w_up, w_down, flags: int = 0, stream=None) -> None:
    _check(lib().moe_expert_ffn_ex(ctypes.byref(heap), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                   int(flags), _stream(stream)), "moe_expert_ffn_ex")


def moe_combine_ex(heap: SymHeapDesc, expert_out, idx, w, out, flags: int = 0, stream=None) -> None:
    _check(lib().moe_combine_ex(ctypes.byref(heap), _ptr(expert_out), _ptr(idx), _ptr(w), _ptr(out),
                                int(flags), _stream(stream)), "moe_combine_ex")


def moe_combine_fallback_copies() -> int:
    return int(lib().moe_combine_fallback_copies())


def moe_pipeline(heap: SymHeapDesc, logits, x, w_gate, w_up, w_down, idx, w, out,
                 mode: int = 0, stream=None) -> None:
    """mode: SYM_PIPE_FUSED, SYM_PIPE_WEIGHTS_IN_FFN, SYM_PIPE_DEDUP bits (0: staged)."""
    _check(lib().moe_pipeline(ctypes.byref(heap), _ptr(logits), _ptr(x), _ptr(w_gate),
                              _ptr(w_up), _ptr(w_down), _ptr(idx), _ptr(w), _ptr(out),
                              int(mode), _stream(stream)), "moe_pipeline")


def moe_dispatch_layout_noalloc(shape, idx, cnt, recv_off, total_recv, pos, stream=None) -> None:
    """Dispatch layout from the routing indices alone, for callers that cannot
    allocate device memory (its scratch is a library-owned device array)."""
    s = _shape(dict(shape, hidden=shape.get("hidden", 128), inter=shape.get("inter", 128)))
    _check(lib().moe_dispatch_layout_noalloc(ctypes.byref(s), _ptr(idx), _ptr(cnt), _ptr(recv_off),
                                             _ptr(total_recv), _ptr(pos), _stream(stream)),
           "moe_dispatch_layout_noalloc")


def sym_heap_windows(heap: SymHeapDesc) -> list:
    """(offset, bytes) of every window inside a slot, in layout order."""
    n = SYM_HEAP_WINDOWS
    offs, sizes = (_u64 * n)(), (_u64 * n)()
    rc = lib().sym_heap_windows(ctypes.byref(heap), offs, sizes, n)
    if rc < 0:
        raise SymmoeError(rc, "sym_heap_windows")
    return [(int(offs[i]), int(sizes[i])) for i in range(rc)]


def sym_heap_status(heap: SymHeapDesc, clear: bool = False, stream=None) -> int:
    st = _i32()
    _check(lib().sym_heap_status(ctypes.byref(heap), ctypes.byref(st), int(clear), _stream(stream)),
           "sym_heap_status")
    return st.value


# ------------------------------------------------------------------ training through an MoE block
# Tensors in, shapes and strides read from them.  A mismatch raises
# SymmoeError(SYM_EINVAL) before anything is launched.

SYM_BF16, SYM_FP16, SYM_FP32 = 0, 1, 2
SYM_GM_TRANS_W = 1
SYM_GM_ACCUMULATE = 1
SYM_GATE_NONE, SYM_GATE_SIGMOID, SYM_GATE_TANH = 0, 1, 2
SYM_NORM_NO_POST = 1
_DTYPES = {torch.bfloat16: SYM_BF16, torch.float16: SYM_FP16, torch.float32: SYM_FP32}
_GATE_ACTS = {"none": SYM_GATE_NONE, "sigmoid": SYM_GATE_SIGMOID, "tanh": SYM_GATE_TANH}


def _need(ok: bool, where: str, why: str) -> None:
    if not ok:
        e = SymmoeError(SYM_EINVAL, where)
        e.args = (f"{e.args[0]}: {why}",)
        raise e


# These calls are made many times a step on small tensors: the helpers touch
# each tensor attribute once.
def _on_device(where: str, *tensors) -> int:
    """The current device, which every tensor has to be on."""
    dev = torch.cuda.current_device() if torch.cuda.is_initialized() else -2
    for t in tensors:
        if t is not None and not (isinstance(t, torch.Tensor) and t.get_device() == dev):
            _need(False, where, "tensors of the current CUDA device are wanted")
    return dev


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, dev: int):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _rows(t, where: str, dtype=None) -> SymRows:
    """[rows, cols], or [slots, rows, cols] such as a heap's windows."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        slots, slot_stride = 1, 0
        rows, cols = shape
        ld, inner = stride
    elif len(shape) == 3:
        slots, rows, cols = shape
        slot_stride, ld, inner = stride
    else:
        _need(False, where, "rows [R, C] or [slots, R, C] are wanted")
    if dtype is not None and t.dtype != dtype:
        _need(False, where, "tensors of one type are wanted")
    if inner != 1 and cols != 1:
        _need(False, where, "the last dimension has to be contiguous")
    if rows <= 1:
        ld = (cols + 7) // 8 * 8
    return SymRows(t.data_ptr(), ld, slot_stride, rows, slots, cols)


def _per_slot(t, slots: int, n: int, dtype, where: str) -> int:
    """Slot stride of a [slots, n] (or, with one slot, [n]) tensor."""
    _need(t.dtype == dtype and t.shape in ((slots, n), (n,) if slots == 1 else (slots, n)) and
          (n == 1 or t.stride(-1) == 1), where, f"[{slots}, {n}] {dtype} is wanted")
    return t.stride(0) if t.dim() == 2 else 0


def _groups(cnt, off, rows: SymRows, status, where: str) -> SymGroups:
    g = cnt.numel()
    _need(g > 0 and rows.slots > 0 and g % rows.slots == 0, where, "the slots have equally many groups")
    each = g // rows.slots
    cs = _per_slot(cnt, rows.slots, each, torch.int32, where)
    os_ = _per_slot(off, rows.slots, each, torch.int32, where)
    _need(status is None or (status.dtype == torch.int32 and status.numel() >= 1), where, "status is an int32 word")
    return SymGroups(cnt.data_ptr(), off.data_ptr(), cs, os_, 0 if status is None else status.data_ptr(), g,
                     rows.slots, 0, 0)


def _matrices(w, groups: int, shape, where: str):
    _need(w.dim() == 3 and tuple(w.shape) == (groups, *shape) and (w.shape[2] == 1 or w.stride(2) == 1), where,
          f"one matrix for each group, [{groups}, {shape[0]}, {shape[1]}], is wanted")
    return w.stride(0), (w.stride(1) if w.shape[1] > 1 else (w.shape[2] + 7) // 8 * 8)


def moe_grouped_matmul(x, w, cnt, off, out, trans_w: bool = False, status=None, stream=None) -> None:
    """out[r] = w[e] @ x[r] for the rows r of group e (w [E, F, C]), or with
    trans_w x[r] @ w[e] (w [E, C, F]: on a forward product's weights, its data
    gradient).  x [R, C] or [slots, R, C]; cnt, off: int32 rows and first row
    of each group, [E] or [slots, E / slots]; bf16 or fp16."""
    where = "moe_grouped_matmul"
    dev = _on_device(where, x, w, cnt, off, out, status)
    rx, ro = _rows(x, where), _rows(out, where, x.dtype)
    g = _groups(cnt, off, rx, status, where)
    _need(w.dtype == x.dtype, where, "x, w and out have one type")
    ws, wl = _matrices(w, g.groups, (rx.cols, ro.cols) if trans_w else (ro.cols, rx.cols), where)
    _check(lib().moe_grouped_matmul(ctypes.byref(g), _DTYPES.get(x.dtype, -1), ctypes.byref(rx), w.data_ptr(), ws, wl,
                                    SYM_GM_TRANS_W if trans_w else 0, ctypes.byref(ro), _stream_of(stream, dev)), where)


def moe_grouped_wgrad(dy, x, cnt, off, dw, accumulate: bool = False, status=None, stream=None) -> None:
    """dw[e] = dy_e^T x_e over the rows of group e (added to dw with
    accumulate); dw [E, F, C] of the inputs' type or float32."""
    where = "moe_grouped_wgrad"
    dev = _on_device(where, dy, x, cnt, off, dw, status)
    ry, rx = _rows(dy, where, x.dtype), _rows(x, where)
    g = _groups(cnt, off, rx, status, where)
    ws, wl = _matrices(dw, g.groups, (ry.cols, rx.cols), where)
    _check(lib().moe_grouped_wgrad(ctypes.byref(g), _DTYPES.get(x.dtype, -1), ctypes.byref(ry), ctypes.byref(rx),
                                   dw.data_ptr(), ws, wl, _DTYPES.get(dw.dtype, -1),
                                   SYM_GM_ACCUMULATE if accumulate else 0, _stream_of(stream, dev)), where)


def _row_words(t, rows: SymRows, dtype, where: str):
    """(address, slot stride) of one word for each row, or none."""
    return (None, 0) if t is None else (t.data_ptr(), _per_slot(t, rows.slots, rows.rows, dtype, where))


def _totals(total, rows: SymRows, where: str):
    if total is None:
        return None, 0
    n = rows.slots
    _need(total.dtype == torch.int32 and (total.shape in ((n,), (n, 1)) or n == 1 and total.dim() == 0), where,
          "total is one int32 for each slot, [slots] or [slots, 1]")
    return total.data_ptr(), (total.stride(0) if n > 1 else 0)


def moe_swiglu_rows(g, u, h, row_w=None, total=None, stream=None) -> None:
    """h = row_w * silu(g) * u; row_w float32 [R] or [slots, R]; total: int32
    rows to do in each slot (all without it)."""
    where = "moe_swiglu_rows"
    dev = _on_device(where, g, u, h, row_w, total)
    rg, ru, rh = _rows(g, where), _rows(u, where, g.dtype), _rows(h, where, g.dtype)
    rw, rws = _row_words(row_w, rg, torch.float32, where)
    tt, ts = _totals(total, rg, where)
    _check(lib().moe_swiglu_rows(_DTYPES.get(g.dtype, -1), ctypes.byref(rg), ctypes.byref(ru), rw, rws, tt, ts,
                                 ctypes.byref(rh), _stream_of(stream, dev)), where)


def moe_swiglu_rows_bwd(g, u, dh, dg, du, row_w=None, d_row_w=None, total=None, stream=None) -> None:
    """Gradients of moe_swiglu_rows: dg, du and, where given, d_row_w."""
    where = "moe_swiglu_rows_bwd"
    dev = _on_device(where, g, u, dh, dg, du, row_w, d_row_w, total)
    rg, ru, rh = _rows(g, where), _rows(u, where, g.dtype), _rows(dh, where, g.dtype)
    r1, r2 = _rows(dg, where, g.dtype), _rows(du, where, g.dtype)
    rw, rws = _row_words(row_w, rg, torch.float32, where)
    dw, dws = _row_words(d_row_w, rg, torch.float32, where)
    tt, ts = _totals(total, rg, where)
    _check(lib().moe_swiglu_rows_bwd(_DTYPES.get(g.dtype, -1), ctypes.byref(rg), ctypes.byref(ru), ctypes.byref(rh),
                                     rw, rws, tt, ts, ctypes.byref(r1), ctypes.byref(r2), dw, dws, _stream_of(stream, dev)),
           where)


def moe_dropout(x, y, p: float, seed: int, offset: int = 0, residual=None, stream=None) -> None:
    """y = residual + x * keep / (1 - p); element i is kept by word i of the
    counter-based stream (seed, offset).  On y's gradient the same call is the
    backward pass."""
    where = "moe_dropout"
    dev = _on_device(where, x, y, residual)
    rx, ry = _rows(x, where), _rows(y, where, x.dtype)
    rr = None if residual is None else ctypes.byref(_rows(residual, where, x.dtype))
    _check(lib().moe_dropout(_DTYPES.get(x.dtype, -1), ctypes.byref(rx), rr, ctypes.byref(ry), p, seed, offset,
                             _stream_of(stream, dev)), where)


def _plain(t, rows: int, cols: int, dtype, where: str):
    """(address, row stride) of a [rows, cols] tensor; (0, 0) for none."""
    if t is None:
        return 0, 0
    stride = t.stride()
    if t.shape != (rows, cols) or t.dtype != dtype or (stride[1] != 1 and cols != 1):
        _need(False, where, f"[{rows}, {cols}] with contiguous rows, of one type, is wanted")
    return t.data_ptr(), stride[0] if rows > 1 else (cols + 7) // 8 * 8


def _vector(t, n: int, dtype, where: str) -> int:
    if t is None:
        return 0
    if t.shape != (n,) or t.dtype != dtype or (n > 1 and t.stride()[0] != 1):
        _need(False, where, f"[{n}] {dtype} is wanted")
    return t.data_ptr()


def _block(where: str, dt, rows: int, cols: int, x, o, w_post, gate, gate_act, scale, p, seed, offset, w_pre, y, h,
           rstd_post, rstd_pre, post_norm, eps) -> SymBlockNorm:
    xp, xl = _plain(x, rows, cols, dt, where)
    op, ol = _plain(o, rows, cols, dt, where)
    yp, yl = _plain(y, rows, cols, dt, where)
    hp, hl = _plain(h, rows, cols, dt, where)
    gates = 0 if gate is None else gate.shape[0]
    # (an empty tensor has no address, which would read as no gate)
    _need(gate is None or gates > 0 or rows == 0, where, "a gate has at least one row")
    gp, gl = _plain(gate, gates, cols, dt, where)
    return SymBlockNorm(rows, cols, _DTYPES.get(dt, -1), xp, op, _vector(w_post, cols, dt, where), gp,
                        _vector(w_pre, cols, dt, where), yp, hp, _vector(rstd_post, rows, torch.float32, where),
                        _vector(rstd_pre, rows, torch.float32, where), xl, ol, gl, yl, hl, gates,
                        _GATE_ACTS.get(gate_act, -1), 0 if post_norm else SYM_NORM_NO_POST, scale, eps, p, seed, offset)


def moe_block_norm(x, o=None, w_post=None, gate=None, gate_act="none", scale: float = 1.0, p: float = 0.0,
                   seed: int = 0, offset: int = 0, y=None, w_pre=None, h=None, rstd_post=None, rstd_pre=None,
                   post_norm: bool = True, eps: float = 1e-6, stream=None) -> None:
    """y = x + scale * drop(act(gate) * norm(o) * w_post), h = norm(y) * w_pre,
    in one pass over the rows [R, C].  Without o only h = norm(x) * w_pre;
    without h only y; post_norm False: o enters as it is.  gate [G, C]: row r
    uses gate row r // (R / G), through gate_act "none", "sigmoid" or "tanh".
    rstd_post, rstd_pre: float32 [R], kept for the backward."""
    where = "moe_block_norm"
    dev = _on_device(where, x, o, w_post, gate, y, w_pre, h, rstd_post, rstd_pre)
    _need(x.dim() == 2, where, "x is [rows, cols]")
    a = _block(where, x.dtype, *x.shape, x, o, w_post, gate, gate_act, scale, p, seed, offset, w_pre, y, h, rstd_post,
               rstd_pre, post_norm, eps)
    _check(lib().moe_block_norm(ctypes.byref(a), _stream_of(stream, dev)), where)


def moe_block_norm_workspace(rows: int, cols: int, gate_rows: int = 0) -> int:
    """Workspace bytes of moe_block_norm_bwd."""
    out = _u64()
    _check(lib().moe_block_norm_workspace(rows, cols, gate_rows, ctypes.byref(out)), "moe_block_norm_workspace")
    return out.value


def moe_block_norm_bwd(dy=None, dh=None, y=None, o=None, w_post=None, gate=None, gate_act="none", scale: float = 1.0,
                       p: float = 0.0, seed: int = 0, offset: int = 0, w_pre=None, rstd_post=None, rstd_pre=None,
                       post_norm: bool = True, dx=None, do=None, dw_pre=None, dw_post=None, dgate=None, work=None,
                       stream=None) -> None:
    """Gradients of moe_block_norm from dy (of y) and dh (of h), with the
    forward's arguments and its y, rstd_post and rstd_pre.  Every output may
    be left out.  work: a uint8 tensor of moe_block_norm_workspace bytes."""
    where = "moe_block_norm_bwd"
    dev = _on_device(where, dy, dh, y, o, w_post, gate, w_pre, rstd_post, rstd_pre, dx, do, dw_pre, dw_post, dgate, work)
    lead = dy if dy is not None else dh
    _need(lead is not None and lead.dim() == 2, where, "dy or dh, [rows, cols], is wanted")
    (rows, cols), dt = lead.shape, lead.dtype
    a = _block(where, dt, rows, cols, None, o, w_post, gate, gate_act, scale, p, seed, offset, w_pre, y, None,
               rstd_post, rstd_pre, post_norm, 0.0)
    dyp, dyl = _plain(dy, rows, cols, dt, where)
    dhp, dhl = _plain(dh, rows, cols, dt, where)
    dxp, dxl = _plain(dx, rows, cols, dt, where)
    dop, dol = _plain(do, rows, cols, dt, where)
    dgp, dgl = _plain(dgate, a.gate_rows, cols, dt, where)
    g = SymBlockNormGrad(dyp, dhp, dxp, dop, _vector(dw_pre, cols, dt, where), _vector(dw_post, cols, dt, where), dgp,
                         dyl, dhl, dxl, dol, dgl)
    if work is not None:
        _need(work.is_contiguous(), where, "work is contiguous")
        g.work, g.work_bytes = work.data_ptr(), work.numel() * work.element_size()
    _check(lib().moe_block_norm_bwd(ctypes.byref(a), ctypes.byref(g), _stream_of(stream, dev)), where)


# ------------------------------------------------------------------ heap owner

class SymHeap:
    """One symmetric heap in a torch-owned device allocation, with views.

    Every view is a slice of ``self.buf`` (no copy); slot ``d``'s copy of a
    window starts at ``d * per_rank_size + off``.
    """

    def __init__(self, shape: dict, device="cuda", align: int = 0):
        self.shape = dict(shape)
        prs, total = sym_heap_bytes(shape, align)
        # zeroed once: the status word and the fused-kernel counters start at 0
        self.buf = torch.zeros(total + 256, dtype=torch.uint8, device=device)
        pad = (-self.buf.data_ptr()) % 256
        self.buf = self.buf[pad:pad + total]
        self.desc = sym_heap_init(shape, self.buf.data_ptr(), total, align)

    # raw window views --------------------------------------------------
    def _win(self, slot: int, off: int, nbytes: int, dtype) -> torch.Tensor:
        base = slot * self.desc.per_rank_size + off
        return self.buf[base:base + nbytes].view(dtype)

    @property
    def cap(self) -> int:
        return self.desc.cap

    def recv_x(self, d: int) -> torch.Tensor:
        H = self.shape["hidden"]
        return self._win(d, self.desc.off_recv_x, self.cap * H * 2, torch.bfloat16).view(self.cap, H)

    def y(self, d: int) -> torch.Tensor:
        H = self.shape["hidden"]
        return self._win(d, self.desc.off_y, self.cap * H * 2, torch.bfloat16).view(self.cap, H)

    def h(self, d: int) -> torch.Tensor:
        I = self.shape["inter"]
        return self._win(d, self.desc.off_h, self.cap * I * 2, torch.bfloat16).view(self.cap, I)

    def recv_pair(self, d: int) -> torch.Tensor:
        return self._win(d, self.desc.off_recv_pair, self.cap * 4, torch.int32)

    def recv_w(self, d: int) -> torch.Tensor:
        return self._win(d, self.desc.off_recv_w, self.cap * 4, torch.float32)

    def pos(self, d: int) -> torch.Tensor:
        T, k = self.shape["tokens_per_slot"], self.shape["topk"]
        return self._win(d, self.desc.off_pos, T * k * 4, torch.int32).view(T, k)

    def cnt(self, d: int) -> torch.Tensor:
        el = self.shape["num_experts"] // self.shape["world"]
        return self._win(d, self.desc.off_cnt, el * 4, torch.int32)

    def recv_off(self, d: int) -> torch.Tensor:
        el = self.shape["num_experts"] // self.shape["world"]
        return self._win(d, self.desc.off_recv_off, el * 4, torch.int32)

    def total_recv(self, d: int) -> torch.Tensor:
        return self._win(d, self.desc.off_total, 4, torch.int32)

    def ready(self, d: int) -> torch.Tensor:
        return self._win(d, self.desc.off_ready, self.desc.num_ready * 4, torch.int32)

    def combine_in_view(self) -> torch.Tensor:
        """Expert-output window as [W, cap, H] (strided by the slot size);
        its data_ptr is the one moe_combine treats as zero-copy."""
        H = self.shape["hidden"]
        W = self.shape["world"]
        base = self.buf[self.desc.off_y:].view(torch.bfloat16)
        return base.as_strided((W, self.cap, H), (self.desc.per_rank_size // 2, H, 1))

    def window(self, name: str) -> torch.Tensor:
        """A per-slot window as one tensor over all slots (strided by the slot
        size, zero copy), for the calls that take rows or groups: "recv_x",
        "y" [W, cap, H]; "h" [W, cap, I]; "recv_w" [W, cap]; "cnt", "recv_off"
        [W, E/W]; "total" [W]."""
        W, H, I = self.shape["world"], self.shape["hidden"], self.shape["inter"]
        el, cap = self.shape["num_experts"] // W, self.cap
        tail, dtype, off = {"recv_x": ((cap, H), torch.bfloat16, self.desc.off_recv_x),
                            "y": ((cap, H), torch.bfloat16, self.desc.off_y),
                            "h": ((cap, I), torch.bfloat16, self.desc.off_h),
                            "recv_w": ((cap,), torch.float32, self.desc.off_recv_w),
                            "cnt": ((el,), torch.int32, self.desc.off_cnt),
                            "recv_off": ((el,), torch.int32, self.desc.off_recv_off),
                            "total": ((), torch.int32, self.desc.off_total)}[name]
        base = self.buf[off:].narrow(0, 0, (self.buf.numel() - off) // 4 * 4).view(dtype)
        inner = (tail[1], 1) if len(tail) == 2 else (1,) * len(tail)
        return base.as_strided((W, *tail), (self.desc.per_rank_size // base.element_size(), *inner))

    def status_word(self) -> torch.Tensor:
        """The heap's status word as a tensor (for the grouped products' status)."""
        return self._win(0, self.desc.off_status, 4, torch.int32)

    def status(self, clear: bool = False, stream=None) -> int:
        return sym_heap_status(self.desc, clear, stream)

    def guard_bands(self) -> list:
        """(start, length) byte ranges of ``self.buf`` that no call touches:
        the bands after every window of every slot."""
        wins = sym_heap_windows(self.desc)
        prs = self.desc.per_rank_size
        ends = [o + b for o, b in wins]
        starts = [o for o, _ in wins[1:]] + [prs]
        return [(d * prs + e, s - e) for d in range(self.shape["world"]) for e, s in zip(ends, starts)]

    # calls -----------------------------------------------------------------
    def route_topk(self, logits, idx, w, stream=None):
        moe_route_topk(self.desc, logits, idx, w, stream)

    def router_logits(self, x, w_router, logits, stream=None):
        moe_router_logits(self.desc, x, w_router, logits, stream)

    def router_splits(self) -> int:
        return moe_router_splits(self.desc)

    def dispatch(self, x, idx, w, dedup=False, fp8=False, stream=None):
        moe_dispatch_ex(self.desc, x, idx, w,
                        (SYM_DISPATCH_DEDUP if dedup else 0) | (SYM_DISPATCH_FP8 if fp8 else 0), stream)

    def expert_ffn(self, wg, wu, wd, weighted_rows=False, stream=None):
        moe_expert_ffn_ex(self.desc, wg, wu, wd, SYM_FFN_WEIGHTED_ROWS if weighted_rows else 0, stream)

    def combine(self, idx, w, out, expert_out=None, unweighted=False, stream=None):
        moe_combine_ex(self.desc, expert_out, idx, w, out, SYM_COMBINE_UNWEIGHTED if unweighted else 0,
                       stream)

    def pipeline(self, logits, x, wg, wu, wd, idx, w, out, fused=0, weights_in_ffn=False, dedup=False,
                 fp8=False, stream=None):
        mode = ((SYM_PIPE_FUSED if fused else 0) | (SYM_PIPE_WEIGHTS_IN_FFN if weights_in_ffn else 0)
                | (SYM_PIPE_DEDUP if dedup else 0) | (SYM_PIPE_FP8 if fp8 else 0))
        moe_pipeline(self.desc, logits, x, wg, wu, wd, idx, w, out, mode, stream)

    def gemm_a2a(self, x, w, fused=False, stream=None):
        sym_gemm_a2a(self.desc, x, w, SYM_LA_FUSED if fused else 0, stream)

    def a2a_gemm(self, z, w, fused=False, copy_engines=False, stream=None):
        mode = (SYM_LA_FUSED | (SYM_LA_COPY_ENGINES if copy_engines else 0)) if fused else 0
        sym_a2a_gemm(self.desc, z, w, mode, stream)


lib()  # fail loudly at import if the CUDA library is missing
