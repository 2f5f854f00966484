"""moe_expert_amd -- block-quantized weight x q8_1 activation products on MI355X (gfx950).

A thin ctypes binding over ``libqmm.so`` (the C ABI declared in include/qmm.h).  Every entry
point below only marshals arguments: it takes torch tensors that already live on the GPU,
checks that each one is a contiguous tensor of the expected dtype on the same GPU and holds at
least the bytes the call reads or writes (``ValueError`` otherwise, before anything is launched:
the library trusts the sizes it is given), passes the device pointers and the current HIP stream
to the library and raises ``QmmError`` on a non-zero status.  All arithmetic runs in the
library's HIP kernels; there is no CPU fallback, and a missing library raises at first use.

Names follow the C ABI: ``qmm_quantize_q8_1``, ``qmm_dequant_f16``, ``qgemv_dense``,
``qgemv_dense_f32``, ``qmm_debug_block_sums``, ``qgemv_grouped_experts``,
``qgemm_prefill_experts`` (and the measurement hooks ``qmm_debug_stream_read``,
``qmm_debug_mfma_loop``); between the products ``qmm_rmsnorm``, ``qmm_dequantize_q8_1``,
``qmm_moe_route``, ``qmm_moe_dispatch`` and ``qmm_lora``, and over a paged key-value cache (``KvCache``)
``qmm_kv_write``, ``qmm_kv_read`` and ``qmm_kv_attend``, which also take row-strided views of
float32, float16 or bfloat16 tensors where their docstrings say so.  What these make anew on a given
stream is that stream's memory: as with torch's own tensors, ``record_stream`` it where work of another
stream may outlive it.
"""
from __future__ import annotations

import ctypes as C
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmm.so")

QMM_Q8_0, QMM_IQ4_NL, QMM_CB3, QMM_F16 = 1, 2, 3, 4
QMM_FLAG_DEBUG_INTERMEDIATES = 1
QMM_TYPE_F32, QMM_TYPE_F16, QMM_TYPE_BF16 = 1, 2, 3
QMM_SCORE_SOFTMAX, QMM_SCORE_SIGMOID = 0, 1
QMM_ROUTE_RENORM = 1
QMM_ESPACE = -5
BLOCK_VALUES = {QMM_Q8_0: 32, QMM_IQ4_NL: 32, QMM_CB3: 256, QMM_F16: 1}
BLOCK_BYTES = {QMM_Q8_0: 34, QMM_IQ4_NL: 18, QMM_CB3: 110, QMM_F16: 2}
Q8_1_BYTES = 36
GRID_BYTES = 2048

_P, _I64, _I32, _U32, _U64, _SZ, _F32 = (C.c_void_p, C.c_int64, C.c_int, C.c_uint, C.c_uint64, C.c_size_t,
                                         C.c_float)
SIGNATURES = {
    "qmm_version": (_I32, []),
    "qmm_status_str": (C.c_char_p, [_I32]),
    "qmm_row_bytes": (_I64, [_I32, _I64]),
    "qmm_quantize_q8_1": (_I32, [_P, _I64, _I32, _I64, _P, _P]),
    "qmm_dequant_f16": (_I32, [_I32, _P, _P, _I64, _I64, _P, _I64, _P]),
    "qgemv_dense": (_I32, [_I32, _P, _P, _I64, _I64, _P, _I32, _P, _I64, _P]),
    "qgemv_dense_f32": (_I32, [_I32, _P, _P, _I64, _I64, _P, _I32, _P, _I64, _P]),
    "qmm_debug_block_sums": (_I32, [_I32, _P, _P, _I64, _I64, _P, _I32, _P, _P]),
    "qmm_debug_stream_read": (_I32, [_P, _U64, _P, _I32, _I32, _I32, _P]),
    "qmm_debug_mfma_loop": (_I32, [_P, _I32, _I32, _P]),
    "qgemv_grouped_experts_workspace": (_SZ, [_I64, _I32, _U32]),
    "qgemv_grouped_experts": (_I32, [_I32, _P, _P, _I64, _I32, _P, _I64, _I32, _P, _I64, _I64, _P, _I32,
                                     _P, _P, _I32, _P, _I32, _P, _P, _SZ, _U32, _P]),
    "qgemv_grouped_experts_noalloc_max_bytes": (_SZ, []),
    "qgemv_grouped_experts_noalloc": (_I32, [_I32, _P, _P, _I64, _I32, _P, _I64, _I32, _P, _I64, _I64, _P, _I32,
                                             _P, _P, _I32, _P, _I32, _P, _P]),
    "qmm_moe_combine": (_I32, [_P, _I64, _I64, _P, _P, _I64, _I32, _P, _I64, _P]),
    "qmm_pack_planes": (_I32, [_I32, _P, _I64, _I64, _P, _P]),
    "qmm_planes_alloc": (_I32, [_I32, _P, _I64, _I64, C.POINTER(C.c_void_p), _P]),
    "qmm_planes_release": (_I32, [_P]),
    "qgemv_planes": (_I32, [_I32, _P, _I64, _I64, _P, _I32, _P, _I64, _P]),
    "qgemm_dense": (_I32, [_I32, _P, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "qgemm_prefill_experts_q8_workspace": (_SZ, [_I32, _I64, _I64, _I64, _I64, _U32]),
    "qgemm_prefill_experts_q8": (_I32, [_I32, _P, _P, _I64, _I32, _P, _I64, _I32, _I64, _I64, _P, _I64,
                                        _P, _P, _I64, _P, _P, _SZ, _U32, _P]),
    "qgemm_prefill_experts_workspace": (_SZ, [_I32, _I64, _I64, _U32]),
    "qgemm_prefill_experts": (_I32, [_I32, _P, _P, _I64, _I32, _P, _I64, _I32, _I64, _I64, _P, _I64,
                                     _P, _P, _I64, _P, _P, _SZ, _U32, _P]),
    "qmm_rmsnorm": (_I32, [_I32, _P, _I64, _I32, _P, _I64, _P, _I64, _P, _F32, _I64, _I64, _I32, _P, _I64, _P, _P]),
    "qmm_dequantize_q8_1": (_I32, [_P, _I64, _I64, _I32, _P, _I64, _P]),
    "qmm_moe_route": (_I32, [_I32, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _U32, _P]),
    "qmm_moe_dispatch_workspace": (_SZ, [_I64, _I32, _I32]),
    "qmm_moe_dispatch": (_I32, [_P, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "qmm_lora_workspace": (_SZ, [_I64, _I32]),
    "qmm_lora": (_I32, [_I32, _P, _I64, _I64, _I64, _P, _P, _P, _P, _I32, _I32, _P, _P, _I32, _P, _I64, _P, _I64, _I64,
                        _P, _SZ, _P]),
    "qmm_kv_write": (_I32, [_P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _I64, _P, _I64, _I64, _P]),
    "qmm_kv_read": (_I32, [_P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _I64, _P, _I64, _I64, _P]),
    "qmm_kv_attend_workspace": (_SZ, [_P, _I64, _I32, _I32, _I64]),
    "qmm_kv_attend": (_I32, [_P, _P, _I64, _I64, _P, _P, _I32, _I32, _P, _I64, _I64, _I32, _F32, _I64, _I32, _P, _I64, _P,
                             _P, _SZ, _P]),
}

_lib = None


class QmmError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({status_str(status)})")
        self.status = status


def lib():
    """Load libqmm.so from the package directory (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m moe_expert_amd.build`")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().qmm_status_str(status).decode()


def row_bytes(wtype: int, k: int) -> int:
    return int(lib().qmm_row_bytes(wtype, k))


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    if stream is not None:
        return C.c_void_p(stream)
    import torch
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise QmmError(fn, rc)


# ------------------------------------------------------------------ argument checks
#
# The C library takes plain pointers and sizes and cannot see the allocations behind them, so
# every tensor is checked here against what the call will touch.

_DTYPES = {}


def _dtypes(kind):
    if not _DTYPES:
        import torch
        _DTYPES.update({"u8": (torch.uint8,), "f32": (torch.float32,), "i32": (torch.int32,),
                        "f16": tuple(d for d in (torch.float16, torch.int16, getattr(torch, "uint16", None))
                                     if d is not None)})
    return _DTYPES[kind]


def _nbytes(t) -> int:
    return int(t.numel()) * int(t.element_size())


def _need(t, name, kind, nbytes, device=None):
    """t must be a contiguous GPU tensor of dtype `kind` (u8, f32, i32, f16: any 2-byte type), on
    `device` when given, holding at least `nbytes` bytes."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in _dtypes(kind):
        raise ValueError(f"{name} must have dtype {kind}, not {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if _nbytes(t) < nbytes:
        raise ValueError(f"{name} holds {_nbytes(t)} bytes; the call touches {nbytes}")
    return t


def _block_multiple(wtype, k, name="k"):
    if wtype not in BLOCK_VALUES:
        raise ValueError(f"unknown weight format {wtype}")
    if k < 1 or k % BLOCK_VALUES[wtype]:
        raise ValueError(f"{name}={k} is not a positive multiple of {BLOCK_VALUES[wtype]}")
    return (k // BLOCK_VALUES[wtype]) * BLOCK_BYTES[wtype]


def _grid_arg(wtype, grid, device, name="grid"):
    if wtype == QMM_CB3 or grid is not None:
        _need(grid, name, "u8", GRID_BYTES, device)
    return grid


def _out(t, name, kind, nbytes, device, shape, dtype):
    """A caller-supplied output (checked) or a new one of `shape`."""
    import torch
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _need(t, name, kind, nbytes, device)


# ------------------------------------------------------------------ entry points

def qmm_quantize_q8_1(x, out=None, stream=None):
    """x: float32 [ncols, k] (GPU) -> uint8 [ncols, k/32*36] q8_1 blocks."""
    import torch
    if getattr(x, "dim", lambda: 0)() == 1:
        x = x.view(1, -1)
    if getattr(x, "dim", lambda: 0)() != 2:
        raise ValueError("x must be [ncols, k]")
    ncols, k = x.shape
    if k < 32 or k % 32:
        raise ValueError(f"k={k} is not a positive multiple of 32")
    _need(x, "x", "f32", ncols * k * 4)
    out = _out(out, "out", "u8", ncols * (k // 32) * Q8_1_BYTES, x.device, (ncols, (k // 32) * Q8_1_BYTES),
               torch.uint8)
    _check("qmm_quantize_q8_1", lib().qmm_quantize_q8_1(_ptr(x), k, ncols, k, _ptr(out), _stream(stream, x.device)))
    return out


def qmm_dequant_f16(wtype, w, nrows, k, grid=None, out=None, ld=None, stream=None):
    """Weight blocks -> binary16 [nrows, ld] (returned as torch.float16)."""
    import torch
    rb = _block_multiple(wtype, k)
    ld = k if ld is None else ld
    if nrows < 1 or ld < k:
        raise ValueError("nrows >= 1 and ld >= k")
    _need(w, "w", "u8", nrows * rb)
    _grid_arg(wtype, grid, w.device)
    out = _out(out, "out", "f16", ((nrows - 1) * ld + k) * 2, w.device, (nrows, ld), torch.float16)
    _check("qmm_dequant_f16", lib().qmm_dequant_f16(wtype, _ptr(w), _ptr(grid), nrows, k, _ptr(out), ld,
                                                   _stream(stream, w.device)))
    return out


def _gemv_common(wtype, w, nrows, k, ncols, grid, ldy, check_w=True):
    rb = _block_multiple(wtype, k)
    if nrows < 1 or ncols < 1:
        raise ValueError("nrows and ncols must be positive")
    ldy = nrows if ldy is None else ldy
    if ldy < nrows:
        raise ValueError("ldy < nrows")
    if check_w:
        _need(w, "w", "u8", nrows * rb)
        _grid_arg(wtype, grid, w.device)
    return ldy


def qgemv_dense(wtype, w, nrows, k, xq, ncols, grid=None, y=None, ldy=None, stream=None):
    """y[c, r] for c < ncols: float32 [ncols, ldy] (ldy defaults to nrows)."""
    import torch
    ldy = _gemv_common(wtype, w, nrows, k, ncols, grid, ldy)
    _need(xq, "xq", "u8", ncols * (k // 32) * Q8_1_BYTES, w.device)
    y = _out(y, "y", "f32", ((ncols - 1) * ldy + nrows) * 4, w.device, (ncols, ldy), torch.float32)
    _check("qgemv_dense", lib().qgemv_dense(wtype, _ptr(w), _ptr(grid), nrows, k, _ptr(xq), ncols, _ptr(y), ldy,
                                           _stream(stream, w.device)))
    return y


def qgemv_dense_f32(wtype, w, nrows, k, x, ncols=1, grid=None, y=None, ldy=None, stream=None):
    """1, 2 or 4 fp32 columns x [ncols, k] quantized to q8_1 inside the kernel: y float32
    [ncols, ldy], bitwise qgemv_dense of qmm_quantize_q8_1(x) (k at most 3072)."""
    import torch
    ldy = _gemv_common(wtype, w, nrows, k, ncols, grid, ldy)
    _need(x, "x", "f32", ncols * k * 4, w.device)
    y = _out(y, "y", "f32", ((ncols - 1) * ldy + nrows) * 4, w.device, (ncols, ldy), torch.float32)
    _check("qgemv_dense_f32", lib().qgemv_dense_f32(wtype, _ptr(w), _ptr(grid), nrows, k, _ptr(x), ncols, _ptr(y),
                                                   ldy, _stream(stream, w.device)))
    return y


def qmm_debug_block_sums(wtype, w, nrows, k, xq, ncols, grid=None, out=None, stream=None):
    """Per-block integer sums int32 [ncols, nrows, k/32]."""
    import torch
    _gemv_common(wtype, w, nrows, k, ncols, grid, None)
    _need(xq, "xq", "u8", ncols * (k // 32) * Q8_1_BYTES, w.device)
    out = _out(out, "out", "i32", ncols * nrows * (k // 32) * 4, w.device, (ncols, nrows, k // 32), torch.int32)
    _check("qmm_debug_block_sums", lib().qmm_debug_block_sums(wtype, _ptr(w), _ptr(grid), nrows, k, _ptr(xq), ncols,
                                                             _ptr(out), _stream(stream, w.device)))
    return out


def qmm_debug_stream_read(p, nbytes, grid, threads=256, unroll=8, out=None, stream=None):
    """Plain streaming read of the first nbytes of device tensor p in one launch of `grid`
    workgroups of `threads` threads, `unroll` 16-byte loads in flight per thread, contiguous runs
    per workgroup (the HBM reference); returns out (uint32 [grid * threads])."""
    import torch
    if grid < 1:
        raise ValueError("grid must be positive")
    _need(p, "p", "u8", nbytes)
    out = _out(out, "out", "i32", grid * threads * 4, p.device, (grid * threads,), torch.int32)
    _check("qmm_debug_stream_read", lib().qmm_debug_stream_read(_ptr(p), nbytes, _ptr(out), grid, threads, unroll,
                                                               _stream(stream, p.device)))
    return out


def qmm_debug_mfma_loop(grid, iters, out=None, device="cuda", stream=None):
    """Register-only fp16 MFMA loop (grid * 4 * 8 * iters * 32768 FLOP); returns out (float
    [grid * 256])."""
    import torch
    if grid < 1 or iters < 1:
        raise ValueError("grid and iters must be positive")
    if out is None:
        out = torch.empty(grid * 256, dtype=torch.float32, device=device)
    _need(out, "out", "f32", grid * 256 * 4)
    _check("qmm_debug_mfma_loop", lib().qmm_debug_mfma_loop(_ptr(out), grid, iters, _stream(stream, out.device)))
    return out


def qgemv_grouped_experts_workspace(inter, nentries, flags=0):
    return int(lib().qgemv_grouped_experts_workspace(inter, nentries, flags))


def _expert_weights(t, name, nexperts, matrix_bytes, device):
    """[nexperts, ...] uint8 expert matrices of at least matrix_bytes each; returns the
    per-expert stride in bytes."""
    if getattr(t, "dim", lambda: 0)() < 1 or t.shape[0] != nexperts:
        raise ValueError(f"{name} must be [{nexperts} experts, ...]")
    _need(t, name, "u8", nexperts * matrix_bytes, device)
    stride = _nbytes(t) // nexperts
    if stride < matrix_bytes:
        raise ValueError(f"{name}: {stride} bytes per expert, one matrix is {matrix_bytes}")
    return stride


def qgemv_grouped_experts(wtype_gu, w_gate, w_up, wtype_down, w_down, hidden, inter, xq, group_expert,
                          group_entry_off, entry_col, grid=None, y=None, ws=None, flags=0, stream=None):
    """Grouped MoE decode.  w_gate / w_up: [nexperts, inter * row_bytes(gu, hidden)] bytes,
    w_down: [nexperts, hidden * row_bytes(down, inter)] bytes, xq: [xq_cols, hidden/32*36] q8_1;
    returns (y [nentries, hidden] float32, ws)."""
    import torch
    if getattr(w_gate, "dim", lambda: 0)() < 1:
        raise ValueError("w_gate must be [nexperts, ...]")
    dev = w_gate.device
    nexperts = int(w_gate.shape[0])
    gu_stride = _expert_weights(w_gate, "w_gate", nexperts, inter * _block_multiple(wtype_gu, hidden, "hidden"), dev)
    if _expert_weights(w_up, "w_up", nexperts, gu_stride, dev) != gu_stride:
        raise ValueError("w_up must have w_gate's shape")
    d_stride = _expert_weights(w_down, "w_down", nexperts, hidden * _block_multiple(wtype_down, inter, "inter"), dev)
    _grid_arg(wtype_gu if wtype_gu == QMM_CB3 else wtype_down, grid, dev)
    col_bytes = (hidden // 32) * Q8_1_BYTES
    _need(xq, "xq", "u8", col_bytes, dev)
    if _nbytes(xq) % col_bytes:
        raise ValueError("xq must hold whole q8_1 columns of width hidden")
    xq_cols = _nbytes(xq) // col_bytes
    ngroups = int(group_expert.numel())
    nentries = int(entry_col.numel())
    _need(group_expert, "group_expert", "i32", 0, dev)
    _need(group_entry_off, "group_entry_off", "i32", (ngroups + 1) * 4, dev)
    _need(entry_col, "entry_col", "i32", 0, dev)
    y = _out(y, "y", "f32", nentries * hidden * 4, dev, (nentries, hidden), torch.float32)
    need = qgemv_grouped_experts_workspace(inter, nentries, flags)
    ws = _out(ws, "ws", "u8", need, dev, (max(need, 16),), torch.uint8)
    _check("qgemv_grouped_experts", lib().qgemv_grouped_experts(
        wtype_gu, _ptr(w_gate), _ptr(w_up), gu_stride, wtype_down, _ptr(w_down), d_stride, nexperts, _ptr(grid),
        hidden, inter, _ptr(xq), xq_cols, _ptr(group_expert), _ptr(group_entry_off), ngroups, _ptr(entry_col),
        nentries, _ptr(y), _ptr(ws), _nbytes(ws), flags, _stream(stream, dev)))
    return y, ws


def qgemv_grouped_experts_noalloc(wtype_gu, w_gate, w_up, wtype_down, w_down, hidden, inter, xq, group_expert,
                                  group_entry_off, entry_col, grid=None, y=None, stream=None):
    """The grouped MoE decode without a workspace: H lives in the library's fixed device array
    (qgemv_grouped_experts_noalloc_max_bytes() bytes per GPU; calls that overlap on one GPU race).
    Arguments as qgemv_grouped_experts; returns y [nentries, hidden] float32."""
    import torch
    if getattr(w_gate, "dim", lambda: 0)() < 1:
        raise ValueError("w_gate must be [nexperts, ...]")
    dev = w_gate.device
    nexperts = int(w_gate.shape[0])
    gu_stride = _expert_weights(w_gate, "w_gate", nexperts, inter * _block_multiple(wtype_gu, hidden, "hidden"), dev)
    if _expert_weights(w_up, "w_up", nexperts, gu_stride, dev) != gu_stride:
        raise ValueError("w_up must have w_gate's shape")
    d_stride = _expert_weights(w_down, "w_down", nexperts, hidden * _block_multiple(wtype_down, inter, "inter"), dev)
    _grid_arg(wtype_gu if wtype_gu == QMM_CB3 else wtype_down, grid, dev)
    col_bytes = (hidden // 32) * Q8_1_BYTES
    _need(xq, "xq", "u8", col_bytes, dev)
    if _nbytes(xq) % col_bytes:
        raise ValueError("xq must hold whole q8_1 columns of width hidden")
    ngroups = int(group_expert.numel())
    nentries = int(entry_col.numel())
    _need(group_expert, "group_expert", "i32", 0, dev)
    _need(group_entry_off, "group_entry_off", "i32", (ngroups + 1) * 4, dev)
    _need(entry_col, "entry_col", "i32", 0, dev)
    y = _out(y, "y", "f32", nentries * hidden * 4, dev, (nentries, hidden), torch.float32)
    _check("qgemv_grouped_experts_noalloc", lib().qgemv_grouped_experts_noalloc(
        wtype_gu, _ptr(w_gate), _ptr(w_up), gu_stride, wtype_down, _ptr(w_down), d_stride, nexperts, _ptr(grid),
        hidden, inter, _ptr(xq), _nbytes(xq) // col_bytes, _ptr(group_expert), _ptr(group_entry_off), ngroups,
        _ptr(entry_col), nentries, _ptr(y), _stream(stream, dev)))
    return y


def qgemm_prefill_experts_workspace(nexperts, inter, nentries, flags=0):
    return int(lib().qgemm_prefill_experts_workspace(nexperts, inter, nentries, flags))


def qgemm_prefill_experts(wtype_gu, w_gate, w_up, wtype_down, w_down, nexperts, hidden, inter, x_f16, sorted_tok,
                          expert_off, y=None, ws=None, flags=0, stream=None):
    """Prefill grouped expert GEMM; returns (y [nentries, hidden] float32, ws)."""
    import torch
    if getattr(x_f16, "dim", lambda: 0)() != 2 or x_f16.shape[1] != hidden:
        raise ValueError("x_f16 must be [ntok, hidden]")
    dev = x_f16.device
    ntok = int(x_f16.shape[0])
    _need(x_f16, "x_f16", "f16", ntok * hidden * 2, dev)
    gu_stride = inter * _block_multiple(wtype_gu, hidden, "hidden")
    d_stride = hidden * _block_multiple(wtype_down, inter, "inter")
    for t, n, s in ((w_gate, "w_gate", gu_stride), (w_up, "w_up", gu_stride), (w_down, "w_down", d_stride)):
        if t is None or int(t.numel()) * int(t.element_size()) != nexperts * s:
            raise ValueError(f"{n} must hold {nexperts} expert matrices of {s} bytes")
        _need(t, n, "u8", nexperts * s, dev)
    nentries = int(sorted_tok.numel())
    _need(sorted_tok, "sorted_tok", "i32", 0, dev)
    _need(expert_off, "expert_off", "i32", (nexperts + 1) * 4, dev)
    y = _out(y, "y", "f32", nentries * hidden * 4, dev, (nentries, hidden), torch.float32)
    need = qgemm_prefill_experts_workspace(nexperts, inter, nentries, flags)
    ws = _out(ws, "ws", "u8", need, dev, (max(need, 16),), torch.uint8)
    _check("qgemm_prefill_experts", lib().qgemm_prefill_experts(
        wtype_gu, _ptr(w_gate), _ptr(w_up), gu_stride, wtype_down, _ptr(w_down), d_stride, nexperts, hidden, inter,
        _ptr(x_f16), ntok, _ptr(sorted_tok), _ptr(expert_off), nentries, _ptr(y), _ptr(ws), _nbytes(ws), flags,
        _stream(stream, dev)))
    return y, ws


def qmm_moe_combine(y, row_idx, weights, out=None, ldo=None, stream=None):
    """Router-weighted sum of each token's expert rows in k order: y float32 [nrows, hidden],
    row_idx int32 [ntok, topk], weights float32 [ntok, topk] -> out float32 [ntok, ldo]."""
    import torch
    if getattr(y, "dim", lambda: 0)() != 2 or getattr(row_idx, "dim", lambda: 0)() != 2:
        raise ValueError("y must be [nrows, hidden] and row_idx [ntok, topk]")
    nrows, hidden = int(y.shape[0]), int(y.shape[1])
    ntok, topk = int(row_idx.shape[0]), int(row_idx.shape[1])
    dev = y.device
    _need(y, "y", "f32", nrows * hidden * 4, dev)
    _need(row_idx, "row_idx", "i32", ntok * topk * 4, dev)
    _need(weights, "weights", "f32", ntok * topk * 4, dev)
    ldo = hidden if ldo is None else ldo
    if ldo < hidden:
        raise ValueError("ldo < hidden")
    out = _out(out, "out", "f32", (max(ntok, 1) - 1) * ldo * 4 + hidden * 4, dev, (ntok, ldo), torch.float32)
    _check("qmm_moe_combine", lib().qmm_moe_combine(_ptr(y), nrows, hidden, _ptr(row_idx), _ptr(weights), ntok, topk,
                                                   _ptr(out), ldo, _stream(stream, dev)))
    return out


def qmm_pack_planes(wtype, w, nrows, k, out=None, stream=None):
    """Q8_0 / IQ4_NL rows repacked into planes (16-block tiles: factor bytes, then scales) in a
    caller-owned uint8 buffer of the blocks' size; returns it."""
    import torch
    if wtype not in (QMM_Q8_0, QMM_IQ4_NL):
        raise ValueError("planes are Q8_0 or IQ4_NL")
    rb = _block_multiple(wtype, k)
    _need(w, "w", "u8", nrows * rb)
    out = _out(out, "out", "u8", nrows * rb, w.device, (nrows, rb), torch.uint8)
    _check("qmm_pack_planes", lib().qmm_pack_planes(wtype, _ptr(w), nrows, k, _ptr(out), _stream(stream, w.device)))
    return out


class Planes:
    """A packed copy owned by the library's allocation (qmm_planes_alloc), freed by release()
    (qmm_planes_release) or when the object is collected."""

    def __init__(self, wtype, w, nrows, k, stream=None):
        if wtype not in (QMM_Q8_0, QMM_IQ4_NL):
            raise ValueError("planes are Q8_0 or IQ4_NL")
        rb = _block_multiple(wtype, k)
        _need(w, "w", "u8", nrows * rb)
        self.wtype, self.nrows, self.k, self.device, self.nbytes = wtype, nrows, k, w.device, nrows * rb
        self.ptr = C.c_void_p()
        _check("qmm_planes_alloc", lib().qmm_planes_alloc(wtype, _ptr(w), nrows, k, C.byref(self.ptr),
                                                          _stream(stream, w.device)))

    def release(self):
        if self.ptr:
            _check("qmm_planes_release", lib().qmm_planes_release(self.ptr))
            self.ptr = C.c_void_p()

    def __del__(self):
        try:
            self.release()
        except Exception:
            pass


def qgemv_planes(wtype, planes, nrows, k, xq, ncols, y=None, ldy=None, stream=None):
    """qgemv_dense on planes (a uint8 tensor from qmm_pack_planes, or a Planes object): y
    float32 [ncols, ldy], bitwise qgemv_dense on the original blocks."""
    import torch
    if isinstance(planes, Planes):
        if (planes.wtype, planes.nrows, planes.k) != (wtype, nrows, k) or not planes.ptr:
            raise ValueError("the packed copy holds another matrix (or was released)")
        dev, ptr = planes.device, planes.ptr
        ldy = _gemv_common(wtype, None, nrows, k, ncols, None, ldy, check_w=False)
    else:
        ldy = _gemv_common(wtype, planes, nrows, k, ncols, None, ldy)
        dev, ptr = planes.device, _ptr(planes)
    _need(xq, "xq", "u8", ncols * (k // 32) * Q8_1_BYTES, dev)
    y = _out(y, "y", "f32", ((ncols - 1) * ldy + nrows) * 4, dev, (ncols, ldy), torch.float32)
    _check("qgemv_planes", lib().qgemv_planes(wtype, ptr, nrows, k, _ptr(xq), ncols, _ptr(y), ldy,
                                             _stream(stream, dev)))
    return y


def qgemm_dense(wtype, w, nrows, k, x_f16, y=None, ldy=None, stream=None):
    """Dense prompt projection y [ntok, ldy] float32 = X16 . W16^T: w Q8_0 / IQ4_NL blocks
    (converted to FP16 in the GEMM) or binary16 [nrows, k] (QMM_F16); x_f16 [ntok, k]."""
    import torch
    if wtype not in (QMM_Q8_0, QMM_IQ4_NL, QMM_F16):
        raise ValueError("dense projections take Q8_0, IQ4_NL or F16 weights")
    rb = _block_multiple(wtype, k)
    if getattr(x_f16, "dim", lambda: 0)() != 2 or x_f16.shape[1] != k:
        raise ValueError("x_f16 must be [ntok, k]")
    ntok = int(x_f16.shape[0])
    ldy = nrows if ldy is None else ldy
    if nrows < 1 or ldy < nrows:
        raise ValueError("nrows >= 1 and ldy >= nrows")
    _need(w, "w", "f16" if wtype == QMM_F16 else "u8", nrows * rb)
    _need(x_f16, "x_f16", "f16", ntok * k * 2, w.device)
    y = _out(y, "y", "f32", (max(ntok, 1) - 1) * ldy * 4 + nrows * 4, w.device, (ntok, ldy), torch.float32)
    _check("qgemm_dense", lib().qgemm_dense(wtype, _ptr(w), nrows, k, _ptr(x_f16), ntok, _ptr(y), ldy,
                                           _stream(stream, w.device)))
    return y


def qgemm_prefill_experts_q8_workspace(nexperts, hidden, inter, ntok, nentries, flags=0):
    return int(lib().qgemm_prefill_experts_q8_workspace(nexperts, hidden, inter, ntok, nentries, flags))


def qgemm_prefill_experts_q8(wtype_gu, w_gate, w_up, wtype_down, w_down, nexperts, hidden, inter, x_f16, sorted_tok,
                             expert_off, y=None, ws=None, flags=0, stream=None):
    """MMQ-style prefill (int8 MFMA, q8_1 activations, SwiGLU + q8_1 of H fused); arguments as
    qgemm_prefill_experts; returns (y [nentries, hidden] float32, ws)."""
    import torch
    if getattr(x_f16, "dim", lambda: 0)() != 2 or x_f16.shape[1] != hidden:
        raise ValueError("x_f16 must be [ntok, hidden]")
    dev = x_f16.device
    ntok = int(x_f16.shape[0])
    _need(x_f16, "x_f16", "f16", ntok * hidden * 2, dev)
    gu_stride = inter * _block_multiple(wtype_gu, hidden, "hidden")
    d_stride = hidden * _block_multiple(wtype_down, inter, "inter")
    for t, n, s in ((w_gate, "w_gate", gu_stride), (w_up, "w_up", gu_stride), (w_down, "w_down", d_stride)):
        if t is None or int(t.numel()) * int(t.element_size()) != nexperts * s:
            raise ValueError(f"{n} must hold {nexperts} expert matrices of {s} bytes")
        _need(t, n, "u8", nexperts * s, dev)
    nentries = int(sorted_tok.numel())
    _need(sorted_tok, "sorted_tok", "i32", 0, dev)
    _need(expert_off, "expert_off", "i32", (nexperts + 1) * 4, dev)
    y = _out(y, "y", "f32", nentries * hidden * 4, dev, (nentries, hidden), torch.float32)
    need = qgemm_prefill_experts_q8_workspace(nexperts, hidden, inter, ntok, nentries, flags)
    ws = _out(ws, "ws", "u8", need, dev, (max(need, 16),), torch.uint8)
    _check("qgemm_prefill_experts_q8", lib().qgemm_prefill_experts_q8(
        wtype_gu, _ptr(w_gate), _ptr(w_up), gu_stride, wtype_down, _ptr(w_down), d_stride, nexperts, hidden, inter,
        _ptr(x_f16), ntok, _ptr(sorted_tok), _ptr(expert_off), nentries, _ptr(y), _ptr(ws), _nbytes(ws), flags,
        _stream(stream, dev)))
    return y, ws


# ------------------------------------------------------------------ between the products
#
# These entry points launch kernels of a few microseconds, so their checks read each tensor's
# attributes once, in the order of cost.

_TYPE_OF = {}


def _types():
    """QMM_TYPE_* by torch dtype."""
    if not _TYPE_OF:
        import torch
        _TYPE_OF.update({torch.float32: QMM_TYPE_F32, torch.float16: QMM_TYPE_F16, torch.bfloat16: QMM_TYPE_BF16})
    return _TYPE_OF


def _matrix(t, name, what):
    """The shape of a two-dimensional GPU tensor."""
    shape = getattr(t, "shape", ())
    if len(shape) != 2:
        raise ValueError(f"{name} must be {what}")
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a GPU tensor")
    return shape


def _rows(t, name, shape, device, bf16=True):
    """t must be a GPU tensor of `shape` and of float32, float16 or (bf16) bfloat16 on `device`, whose
    rows are contiguous and do not overlap (any row stride from the width on); returns its type code
    and row stride."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    code = (_TYPE_OF or _types()).get(t.dtype, 0)
    if not code or (code == QMM_TYPE_BF16 and not bf16):
        raise ValueError(f"{name} has dtype {t.dtype}, which this call does not take")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if t.is_contiguous():
        return code, shape[1]
    ld, step = t.stride()
    if shape[0] <= 1:
        ld = shape[1]  # the one row's stride says nothing
    if (step != 1 and shape[1] > 1) or ld < shape[1]:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return code, ld


def _flat(t, name, dtype, count, device):
    """t must be a contiguous tensor of `dtype` on `device` (a GPU) with at least `count` elements."""
    if t.dtype != dtype or t.numel() < count or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {count} elements on {device}")
    return t


def _vector(t, name, dtype, count, device):
    """The same for a vector of weights, of exactly `count` elements: a longer one is another model's."""
    if t.dtype != dtype or t.numel() != count or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} elements on {device}")
    return t


_CURRENT = None


def _current():
    """(current device index, current stream handle of a device index): torch's direct functions, as
    the Stream object that the public call builds costs as much as a launch; the public calls where
    they are missing."""
    global _CURRENT
    if _CURRENT is None:
        import torch
        torch.cuda.init()
        _CURRENT = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                    getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream))
    return _CURRENT


def _call(fn, device, stream, *args):
    """Call a library function on `device`'s current stream (or the one given)."""
    device_of, stream_of = _CURRENT or _current()
    here = device_of()
    at = here if device.index is None else device.index
    if stream is None:
        stream = stream_of(at)
    if at != here:
        import torch
        with torch.cuda.device(at):
            rc = getattr(lib(), fn)(*args, stream)
    else:
        rc = getattr(lib(), fn)(*args, stream)
    if rc != 0:
        raise QmmError(fn, rc)


def _empty(shape, dtype, device, stream):
    """A new tensor of the memory of the stream it is used on (the current one, or the one given): memory
    that another stream's pending work has given back would still be written by it."""
    import torch
    if stream is None or stream == _current()[1](device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    # an ExternalStream of handle 0 is some stream of torch's pool, not the default one
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _scratch(ws, nbytes, device, stream):
    """A caller's workspace (checked), or a new one."""
    import torch
    if ws is not None:
        return _flat(ws, "ws", torch.uint8, nbytes, device)
    return _empty(max(nbytes, 16), torch.uint8, device, stream)


def qmm_rmsnorm(x, w, eps, res=None, res_out=None, y=None, yq=None, stream=None):
    """Root-mean-square norm of r = x + res (or of x), y = r / sqrt(mean r^2 + eps) * w.

    x, res: [ntok, hidden] float32, float16 or bfloat16 with any row stride; w: float32 [hidden].
    Outputs, at least one: y, a tensor or a dtype for a new one; yq, a uint8 tensor of ntok rows of
    hidden/32*36 bytes or True for a new one (q8_1 of the float32 y, for the decode products);
    res_out, a tensor of res' dtype (of any dtype without res) that takes r, res itself for an
    update in place.  Returns (y, yq, res_out), None for those not asked for."""
    import torch
    shape = ntok, hidden = _matrix(x, "x", "[ntok, hidden]")
    dev = x.device
    if hidden < 1:
        raise ValueError("hidden must be positive")
    if y is None and yq is None and res_out is None:
        raise ValueError("no output asked for")
    xt, ldx = _rows(x, "x", shape, dev)
    _vector(w, "w", torch.float32, hidden, dev)
    rt = ldr = ldro = yt = ldy = 0
    if res is not None:
        rt, ldr = _rows(res, "res", shape, dev)
    if res_out is not None:
        ot, ldro = _rows(res_out, "res_out", shape, dev)
        if rt and ot != rt:
            raise ValueError("res_out must have res' dtype")
        rt = ot
    if y is not None:
        if isinstance(y, torch.dtype):
            y = _empty(shape, y, dev, stream)
        yt, ldy = _rows(y, "y", shape, dev)
    if yq is not None:
        if hidden % 32:
            raise ValueError(f"hidden={hidden} is not a multiple of 32")
        nbytes = ntok * (hidden // 32) * Q8_1_BYTES
        if yq is True:
            yq = _empty((ntok, (hidden // 32) * Q8_1_BYTES), torch.uint8, dev, stream)
        _flat(yq, "yq", torch.uint8, nbytes, dev)
    _call("qmm_rmsnorm", dev, stream, xt, x.data_ptr(), ldx, rt, _addr(res), ldr, _addr(res_out), ldro, w.data_ptr(), eps,
          ntok, hidden, yt, _addr(y), ldy, _addr(yq))
    return y, yq, res_out


def _addr(t):
    return None if t is None else t.data_ptr()


def qmm_dequantize_q8_1(xq, k, out=None, stream=None):
    """The values of q8_1 columns: xq uint8 [ncols, k/32*36] -> out [ncols, k], float32 or float16
    (a tensor with any row stride, a dtype for a new one, None for float32)."""
    import torch
    if k < 32 or k % 32:
        raise ValueError(f"k={k} is not a positive multiple of 32")
    _need(xq, "xq", "u8", 0)
    col = (k // 32) * Q8_1_BYTES
    if _nbytes(xq) % col:
        raise ValueError("xq must hold whole q8_1 columns of width k")
    ncols, dev = _nbytes(xq) // col, xq.device
    if out is None or isinstance(out, torch.dtype):
        out = _empty((ncols, k), out or torch.float32, dev, stream)
    ot, ldo = _rows(out, "out", (ncols, k), dev, bf16=False)
    _call("qmm_dequantize_q8_1", dev, stream, xq.data_ptr(), k, ncols, ot, out.data_ptr(), ldo)
    return out


def qmm_moe_route(logits, topk, score=QMM_SCORE_SOFTMAX, bias=None, ngroups=1, topk_groups=1, group_top=1, renorm=True,
                  scale=1.0, ids=None, weights=None, stream=None):
    """Experts of each token: logits [ntok, nexperts] (float32, float16 or bfloat16, any row stride)
    -> (ids int32 [ntok, topk], weights float32 [ntok, topk]), best first, ties to the lowest expert.

    Scores are the softmax or the sigmoid of the logits; experts are chosen by score + bias (float32
    [nexperts]) among the topk_groups best of ngroups runs of experts, a run rated by the sum of its
    group_top best; weights are the chosen scores, divided by their sum if renorm, times scale.
    Experts whose logit or score + bias is -inf or NaN are never chosen (those that only the bias takes
    out count in the softmax); missing choices are id -1, weight 0."""
    import torch
    shape = ntok, nexperts = _matrix(logits, "logits", "[ntok, nexperts]")
    dev = logits.device
    lt, ldl = _rows(logits, "logits", shape, dev)
    if topk < 1 or max(topk, ngroups, topk_groups, group_top) > 0x7FFFFFFF:
        raise ValueError("topk must be positive, and every count an int32")
    if bias is not None:
        _vector(bias, "bias", torch.float32, nexperts, dev)
    if ids is not None:
        _flat(ids, "ids", torch.int32, ntok * topk, dev)
    if weights is not None:
        _flat(weights, "weights", torch.float32, ntok * topk, dev)
    ids = _empty((ntok, topk), torch.int32, dev, stream) if ids is None else ids
    weights = _empty((ntok, topk), torch.float32, dev, stream) if weights is None else weights
    _call("qmm_moe_route", dev, stream, lt, logits.data_ptr(), ldl, _addr(bias), ntok, nexperts, score, ngroups, topk_groups,
          group_top, topk, scale, ids.data_ptr(), weights.data_ptr(), QMM_ROUTE_RENORM if renorm else 0)
    return ids, weights


def qmm_moe_dispatch_workspace(ntok, topk, nexperts):
    return int(lib().qmm_moe_dispatch_workspace(ntok, topk, nexperts))


def qmm_moe_dispatch(ids, nexperts, sorted_tok=None, row_idx=None, expert_off=None, group_expert=None, group_off=None,
                     ws=None, stream=None):
    """The entry lists of a routing: ids int32 [ntok, topk] (an id outside [0, nexperts) adds no
    entry) -> (sorted_tok [ntok*topk], row_idx [ntok, topk], expert_off [nexperts+1],
    group_expert [G], group_off [G+1]) with G = min(nexperts, ntok*topk), all int32:

    qgemm_prefill_experts takes sorted_tok and expert_off, qgemv_grouped_experts group_expert,
    group_off and sorted_tok (as entry_col), qmm_moe_combine row_idx.  Entries are ordered by expert,
    then token, then k; sorted_tok is -1 past the last entry, row_idx -1 where there is none."""
    import torch
    ntok, topk = _matrix(ids, "ids", "[ntok, topk]")
    dev = ids.device
    n = ntok * topk
    g = min(nexperts, n)
    if not 0 < nexperts <= 0x7FFFFFFF or topk < 1:
        raise ValueError("nexperts and topk must be positive, nexperts an int32")
    if (group_expert is None) != (group_off is None):
        raise ValueError("group_expert and group_off go together")
    i32 = torch.int32
    _flat(ids, "ids", i32, n, dev)
    sorted_tok = _empty(n, i32, dev, stream) if sorted_tok is None else _flat(sorted_tok, "sorted_tok", i32, n, dev)
    row_idx = _empty((ntok, topk), i32, dev, stream) if row_idx is None else _flat(row_idx, "row_idx", i32, n, dev)
    if expert_off is None:
        expert_off = _empty(nexperts + 1, i32, dev, stream)
    if group_expert is None:
        group_expert, group_off = _empty(g, i32, dev, stream), _empty(g + 1, i32, dev, stream)
    _flat(expert_off, "expert_off", i32, nexperts + 1, dev)
    _flat(group_expert, "group_expert", i32, g, dev)
    _flat(group_off, "group_off", i32, g + 1, dev)
    ws = _scratch(ws, qmm_moe_dispatch_workspace(ntok, topk, nexperts), dev, stream)
    _call("qmm_moe_dispatch", dev, stream, ids.data_ptr(), ntok, topk, nexperts, sorted_tok.data_ptr(), row_idx.data_ptr(),
          expert_off.data_ptr(), group_expert.data_ptr(), group_off.data_ptr(), ws.data_ptr(), ws.numel())
    return sorted_tok, row_idx, expert_off, group_expert, group_off


def qmm_lora_workspace(ntok, max_rank):
    return int(lib().qmm_lora_workspace(ntok, max_rank))


def qmm_lora(x, a, b, ranks, scales, seg_off, seg_adapter, y, base=None, ws=None, stream=None):
    """Low-rank adapters beside a shared projection: y[t] = base[t] + scales[i] * b[i] (a[i] x[t]),
    i = seg_adapter[s] for the tokens seg_off[s] .. seg_off[s+1]-1 (an i outside the adapters:
    y = base).  base None: y itself, updated in place.

    x: float16 or float32 [ntok, k], rows 16-byte aligned; a: float16 [nadapters, max_rank, k], b:
    float16 [nadapters, nrows, max_rank], of which the first ranks[i] (int32) rows / columns are
    used; scales: float32 [nadapters]; seg_off: int32 [nseg+1]; seg_adapter: int32 [nseg]; y, base:
    float32 [ntok, nrows] with any row stride.  Returns y."""
    import torch
    shape = ntok, k = _matrix(x, "x", "[ntok, k]")
    if len(getattr(a, "shape", ())) != 3 or len(getattr(b, "shape", ())) != 3:
        raise ValueError("a must be [nadapters, max_rank, k], b [nadapters, nrows, max_rank]")
    na, max_rank, ka = a.shape
    nb, nrows, rb = b.shape
    dev = x.device
    if ka != k or nb != na or rb != max_rank:
        raise ValueError("a must be [nadapters, max_rank, k], b [nadapters, nrows, max_rank]")
    xt, ldx = _rows(x, "x", shape, dev, bf16=False)
    _flat(a, "a", torch.float16, 0, dev)
    _flat(b, "b", torch.float16, 0, dev)
    _vector(ranks, "ranks", torch.int32, na, dev)
    _vector(scales, "scales", torch.float32, na, dev)
    nseg = seg_adapter.numel()
    _flat(seg_adapter, "seg_adapter", torch.int32, nseg, dev)
    _flat(seg_off, "seg_off", torch.int32, nseg + 1, dev)
    shape = (ntok, nrows)
    yt, ldy = _rows(y, "y", shape, dev)
    bt, ldb = (yt, ldy) if base is None else _rows(base, "base", shape, dev)
    if yt != QMM_TYPE_F32 or bt != QMM_TYPE_F32:
        raise ValueError("y and base must be float32")
    base = y if base is None else base
    ws = _scratch(ws, qmm_lora_workspace(ntok, max_rank), dev, stream)
    _call("qmm_lora", dev, stream, xt, x.data_ptr(), ldx, ntok, k, a.data_ptr(), b.data_ptr(), ranks.data_ptr(),
          scales.data_ptr(), na, max_rank, seg_off.data_ptr(), seg_adapter.data_ptr(), nseg, base.data_ptr(), ldb,
          y.data_ptr(), ldy, nrows, ws.data_ptr(), ws.numel())
    return y


# ------------------------------------------------------------------ the key-value cache

KV_DIMS = (64, 96, 128, 192, 256)


class _KvStruct(C.Structure):
    """qmm_kv_cache of include/qmm.h."""
    _fields_ = [("ktype", _I32), ("vtype", _I32), ("k", _P), ("v", _P), ("kstride", _I64), ("vstride", _I64), ("npages", _I64),
                ("page_size", _I32), ("nheads", _I32), ("head_dim", _I32)]


class KvCache:
    """A paged key-value cache over two caller-owned tensors, checked once: k of format ktype, v of vtype
    (QMM_F16, QMM_Q8_0 or QMM_IQ4_NL), each [npages, nheads, page_size, row]: float16 with row = head_dim,
    or uint8 with row = row_bytes(type, head_dim) (a page and head's planes of factors and scales; the
    layout is in include/qmm.h).  Pages may lie apart (a view into a larger allocation: the first
    dimension's stride), what is in a page is contiguous.  page_size is a multiple of 16, head_dim 64,
    96, 128, 192 or 256.  Any two formats can be written and read; qmm_kv_attend takes values of at most as many
    bits as the keys.  The object keeps the tensors; it must not outlive a change of their storage."""

    __slots__ = ("ktype", "vtype", "k", "v", "device", "npages", "nheads", "page_size", "head_dim", "width", "_struct", "_ref")

    def __init__(self, ktype, vtype, k, v):
        dims = [self._side(t, kind, name) for t, kind, name in ((k, ktype, "k"), (v, vtype, "v"))]
        if dims[0] != dims[1] or k.device != v.device:
            raise ValueError(f"k and v must hold the same pages, heads and head_dim on one device: {dims[0]}, {dims[1]}")
        self.npages, self.nheads, self.page_size, self.head_dim = dims[0]
        self.ktype, self.vtype, self.k, self.v, self.device = ktype, vtype, k, v, k.device
        self.width = self.nheads * self.head_dim
        # (the stride of a single page says nothing)
        strides = [(t.stride()[0] if self.npages > 1 else t.numel()) * t.element_size() for t in (k, v)]
        self._struct = _KvStruct(ktype, vtype, k.data_ptr(), v.data_ptr(), *strides, self.npages, self.page_size, self.nheads, self.head_dim)
        self._ref = C.addressof(self._struct)

    @staticmethod
    def _side(t, kind, name):
        import torch
        if kind not in (QMM_F16, QMM_Q8_0, QMM_IQ4_NL):
            raise ValueError(f"{name}: caches are QMM_F16, QMM_Q8_0 or QMM_IQ4_NL")
        shape = getattr(t, "shape", ())
        if len(shape) != 4 or min(shape) < 1:
            raise ValueError(f"{name} must be [npages, nheads, page_size, row]")
        if not getattr(t, "is_cuda", False):
            raise ValueError(f"{name} must be a GPU tensor")
        want = torch.float16 if kind == QMM_F16 else torch.uint8
        if t.dtype != want:
            raise ValueError(f"{name} must have dtype {want}, not {t.dtype}")
        npages, nheads, page_size, row = shape
        if page_size % 16 or page_size > 4096 or nheads > 1024 or npages > 0x7FFFFFFF:
            raise ValueError(f"{name}: page_size must be a multiple of 16 up to 4096, nheads at most 1024")
        dim = row if kind == QMM_F16 else row * 32 // BLOCK_BYTES[kind]
        if dim not in KV_DIMS or (kind != QMM_F16 and row != dim // 32 * BLOCK_BYTES[kind]):
            raise ValueError(f"{name}: rows of {row} are not rows of head_dim in {KV_DIMS}")
        st = t.stride()
        inner = (page_size * row, row, 1)
        if any(n > 1 and s != w for n, s, w in zip(shape[1:], st[1:], inner)) or (npages > 1 and st[0] < nheads * page_size * row):
            raise ValueError(f"{name}: what is in a page must be contiguous, and pages must not overlap")
        return npages, nheads, page_size, dim

    @classmethod
    def empty(cls, ktype, vtype, npages, nheads, head_dim, page_size=64, device="cuda"):
        """A new cache of zeros."""
        import torch
        new = [torch.zeros((npages, nheads, page_size, head_dim if kind == QMM_F16 else row_bytes(kind, head_dim)),
                           dtype=torch.float16 if kind == QMM_F16 else torch.uint8, device=device) for kind in (ktype, vtype)]
        return cls(ktype, vtype, *new)


def _kv_sequences(cache, pages, lens, seg_off, ntok):
    """The checks of a call's sequences: (nseq, max_pages, ldpages)."""
    import torch
    i32, dev = torch.int32, cache.device
    if len(getattr(pages, "shape", ())) != 2:
        raise ValueError("pages must be [nseq, max_pages]")
    nseq, width = pages.shape
    if pages.dtype != i32 or pages.device != dev:
        raise ValueError(f"pages must be int32 on {dev}")
    ld = width
    if not pages.is_contiguous():
        ld, step = pages.stride()
        if nseq <= 1:
            ld = width
        if (step != 1 and width > 1) or ld < width:
            raise ValueError("pages must have contiguous rows that do not overlap")
    if width < 1:
        raise ValueError("pages must have a column")
    _vector(lens, "lens", i32, nseq, dev)
    if seg_off is not None:
        _vector(seg_off, "seg_off", i32, nseq + 1, dev)
    elif nseq != ntok:
        raise ValueError(f"{ntok} tokens of {nseq} sequences need seg_off")
    return nseq, width, ld


def qmm_kv_write(cache, pages, lens, k=None, v=None, seg_off=None, stream=None):
    """Writes new tokens' keys and values (either may be None) to a KvCache, quantized per 32 values of a
    head as the cache's format says.

    k, v: [ntok, nheads * head_dim] float32, float16 or bfloat16 (the same), any row stride.  pages: int32
    [nseq, max_pages], each sequence's pages in order (entries it does not need may hold anything); lens:
    int32 [nseq], its length with the new tokens; seg_off: int32 [nseq+1], sequence s has the tokens
    seg_off[s] .. seg_off[s+1]-1, its last positions (None: token s is sequence s's).  A token whose
    position is negative, past the table or on a page outside the cache is not written."""
    x = v if k is None else k
    if x is None:
        raise ValueError("k or v is required")
    ntok = _matrix(x, "k" if k is not None else "v", "[ntok, nheads * head_dim]")[0]
    dev = cache.device
    nseq, width, ldp = _kv_sequences(cache, pages, lens, seg_off, ntok)
    kt = vt = ldk = ldv = 0
    if k is not None:
        kt, ldk = _rows(k, "k", (ntok, cache.width), dev)
    if v is not None:
        vt, ldv = _rows(v, "v", (ntok, cache.width), dev)
        if kt and vt != kt:
            raise ValueError("k and v must have the same dtype")
    _call("qmm_kv_write", dev, stream, cache._ref, pages.data_ptr(), ldp, width, lens.data_ptr(), _addr(seg_off), nseq, kt or vt,
          _addr(k), ldk, _addr(v), ldv, ntok)


def qmm_kv_read(cache, pages, lens, k=None, v=None, seg_off=None, ntok=None, stream=None):
    """Reads positions of a KvCache back: the last seg_off[s+1] - seg_off[s] positions of each sequence
    (None: the last one), in order, into k and v: [ntok, nheads * head_dim] tensors of one of float32,
    float16 and bfloat16 with any row stride, or a dtype for a new one (ntok rows; by default nseq, one of
    each sequence); None for what is not wanted.  Positions that do not exist give rows of zeros; rows of
    no sequence are left alone.  Returns (k, v)."""
    import torch
    dtype, dev = torch.dtype, cache.device
    for t in (v, k):
        if t is not None and not isinstance(t, dtype):
            ntok = _matrix(t, "k and v", "[ntok, nheads * head_dim] or a dtype")[0]
            break
    if ntok is None:
        if seg_off is not None:
            raise ValueError("ntok is required for new tensors of ragged sequences")
        ntok = _matrix(pages, "pages", "[nseq, max_pages]")[0]
    if ntok < 0:
        raise ValueError("ntok must not be negative")
    nseq, width, ldp = _kv_sequences(cache, pages, lens, seg_off, ntok)
    kt = vt = ldk = ldv = 0
    if k is not None:
        if isinstance(k, dtype):
            k = _kv_rows_of(k, "k", (ntok, cache.width), dev, stream)
        kt, ldk = _rows(k, "k", (ntok, cache.width), dev)
    if v is not None:
        if isinstance(v, dtype):
            v = _kv_rows_of(v, "v", (ntok, cache.width), dev, stream)
        vt, ldv = _rows(v, "v", (ntok, cache.width), dev)
        if kt and vt != kt:
            raise ValueError("k and v must have the same dtype")
    if not kt and not vt:
        raise ValueError("k or v is required")
    _call("qmm_kv_read", dev, stream, cache._ref, pages.data_ptr(), ldp, width, lens.data_ptr(), _addr(seg_off), nseq, kt or vt,
          _addr(k), ldk, _addr(v), ldv, ntok)
    return k, v


def _kv_rows_of(dtype, name, shape, device, stream):
    """A new tensor that a read fills."""
    if dtype not in (_TYPE_OF or _types()):
        raise ValueError(f"{name}: {dtype} is not a type that this call writes")
    return _empty(shape, dtype, device, stream)


def qmm_kv_attend_workspace(cache, ntok, nheads, nseq, max_pages):
    """Workspace bytes of qmm_kv_attend for up to these sizes; 0 for sizes it does not take."""
    return int(lib().qmm_kv_attend_workspace(cache._ref, ntok, nheads, nseq, max_pages))


def qmm_kv_attend(q, cache, pages, lens, seg_off=None, scale=None, window=0, out=None, lse=None, ws=None, stream=None):
    """Attention of new tokens over a KvCache that holds their keys and values already (qmm_kv_write).

    q: [ntok, nheads * head_dim] float32, float16 or bfloat16, any row stride, nheads a multiple of the
    cache's; head h reads the cache's head h // (nheads / cache.nheads).  pages, lens, seg_off as
    qmm_kv_write; a token at position p sees the positions j <= p, with window > 0 only j > p - window.
    scale: of the products, 1 / sqrt(head_dim) by default.  out: a tensor like q, of any of the types, or
    a dtype for a new one (default q's; rows of no sequence are left alone); must not be q nor overlap it.  The cache's
    values must hold at most as many bits as its keys.  lse: float32
    [ntok, nheads] or True for a new one: the log of each row's sum of exponentials.  A row that sees no position
    gives zeros and -inf.  ws: qmm_kv_attend_workspace bytes (a call makes its own by default).
    Returns (out, lse)."""
    import torch
    shape = ntok, width = _matrix(q, "q", "[ntok, nheads * head_dim]")
    dev, dim = cache.device, cache.head_dim
    nheads = width // dim
    if width < 1 or width % cache.width:
        raise ValueError(f"q must have a multiple of {cache.width} columns")
    nseq, maxp, ldp = _kv_sequences(cache, pages, lens, seg_off, ntok)
    qt, ldq = _rows(q, "q", shape, dev)
    if out is q:
        raise ValueError("out must not be q")
    if out is None or isinstance(out, torch.dtype):
        if out is not None and out not in (_TYPE_OF or _types()):
            raise ValueError(f"out: {out} is not a type that this call writes")
        out = _empty(shape, out or q.dtype, dev, stream)
    ot, ldo = _rows(out, "out", shape, dev)
    if lse is True:
        lse = _empty((ntok, nheads), torch.float32, dev, stream)
    elif lse is not None:
        _flat(lse, "lse", torch.float32, ntok * nheads, dev)
    if not 0 <= window <= 0x7FFFFFFFFFFFFFFF:
        raise ValueError("window must not be negative")
    own = ws is None
    if own:
        ws = _scratch(None, qmm_kv_attend_workspace(cache, ntok, nheads, nseq, maxp), dev, stream)
    else:
        _flat(ws, "ws", torch.uint8, 16, dev)
    try:
        _call("qmm_kv_attend", dev, stream, cache._ref, pages.data_ptr(), ldp, maxp, lens.data_ptr(), _addr(seg_off), nseq, qt,
              q.data_ptr(), ldq, ntok, nheads, dim ** -0.5 if scale is None else scale, window, ot, out.data_ptr(), ldo, _addr(lse),
              ws.data_ptr(), ws.numel())
    except QmmError as e:
        if e.status != QMM_ESPACE or own:
            raise
        # (the library knows how much it needs: asked for the message alone, a call costs a microsecond)
        _flat(ws, "ws", torch.uint8, qmm_kv_attend_workspace(cache, ntok, nheads, nseq, maxp), dev)
        raise
    return out, lse
