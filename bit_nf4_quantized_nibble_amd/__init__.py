"""QLoRA NF4 linear layer for AMD Instinct MI355X (gfx950).

Thin Python binding over libqlora_nf4.so (C ABI in include/qlora_nf4.h).  This
module only marshals arguments: it checks devices / dtypes / contiguity, passes
raw device pointers and the current HIP stream, and allocates outputs and
workspaces with torch.  Every step of the computation runs in the library's
hand-written HIP kernels; there is no CPU or PyTorch fallback.

Public API (names follow the pages' problem statement):
    quantize(w, block_size=64, double_quant=False, dq_group=256 | "global") -> NF4Weight
    dequantize(q, dtype=torch.bfloat16) -> Tensor [rows, cols]
    linear_fwd_cached(w_cd, x, lora_a, lora_b, alpha, bias=None, save_t=False, rslora=False)
    linear_fwd_noalloc(q, x, lora_a, lora_b, alpha, bias=None, out=None, t_out=None, rslora=False, path="auto")
    linear_fwd(q, x, lora_a, lora_b, alpha, bias=None, save_t=False, rslora=False, path="auto",
               dropout_mask=None, dropout_p=0.0)
    linear_bwd(q, x, dy, lora_a, lora_b, alpha, t_saved=None, need_dx=True, rslora=False, path="auto",
               dropout_mask=None, dropout_p=0.0)
    merge(q, lora_a, lora_b, alpha, rslora=False, out=None) -> Tensor [rows, cols]
    mse_loss_grad(y, target) -> (loss [1] fp32, dy) ; adamw_step(param, grad, m, v, step, ...)
    distill_loss_grad(logits, top_values, top_index, temperature=1.0, weight=None, need_grad=True, dlogits=None,
                      row_kl=None) -> (loss [1] fp32, dlogits or None)
    StackLayer.create(q, a32, b32, dtype) ; stack_train_step(layers, x, target, alpha, step, ...)
    linear_fwd_dropout(q, x, lora_a, lora_b, alpha, p, seed, ...) ; linear_bwd_dropout(q, x, dy, ..., p, seed, ...)
    linear_fwd_gated((q_gate, q_up), x, lora_as, lora_bs, alphas, act="silu", bias=None, save=False) -> h
    linear_bwd_gated((q_gate, q_up), x, dh, lora_as, lora_bs, alphas, pre, act="silu", ...) -> (dX, dAs, dBs)
    quantize_fp8(w) -> Fp8Weight ; linear_fp8(w, x, bias=None)
    quantize_int8(w) -> Int8Weight ; linear_int8(w, x, bias=None) ; linear_int8_experts(w, x, offsets, bias=None)
    workspace_bytes(op, m, rows, cols, r, dtype, flags=0) ; levels()

path: "fused" decodes W inside the GEMM kernels; "dequant" writes W~ (or W~^T for
dX) into the workspace first and runs a dense GEMM; "auto" lets the library pick
(dequantize-then-GEMM for bf16 / f16; "fused" saves the rows x cols copy in the
workspace).  Calls with at most 16 tokens take the decode GEMV either way.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from dataclasses import dataclass
from typing import Optional, Tuple

from . import _lib
from ._lib import QloraError, QloraFp8, QloraInt8, QloraNf4  # noqa: F401

__all__ = ["NF4Weight", "quantize", "dequantize", "linear_fwd", "linear_bwd", "merge", "workspace_bytes",
           "linear_fwd_noalloc", "linear_fwd_cached",
           "levels", "QloraError", "dtype_code", "profile_enable", "profile_read", "mse_loss_grad",
           "adamw_step", "StackLayer", "stack_train_step", "stack_workspace_bytes",
           "linear_fwd_group", "linear_bwd_group", "group_workspace_bytes",
           "Int8Weight", "quantize_int8", "linear_int8", "linear_int8_experts", "int8_workspace_bytes",
           "distill_loss_grad", "linear_fwd_dropout", "linear_bwd_dropout",
           "linear_fwd_gated", "linear_bwd_gated", "gated_workspace_bytes", "Fp8Weight", "quantize_fp8", "linear_fp8",
           "fp8_workspace_bytes"]


def _torch():
    import torch
    return torch


_dtype_codes = {}


def dtype_code(dtype) -> int:
    code = _dtype_codes.get(dtype)
    if code is None:
        code = _dtype_codes[dtype] = _find_dtype_code(dtype)
    return code


def _find_dtype_code(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return _lib.QLORA_F32
    if dtype == torch.bfloat16:
        return _lib.QLORA_BF16
    if dtype == torch.float16:
        return _lib.QLORA_F16
    raise TypeError("unsupported dtype %s (float32, bfloat16 or float16)" % (dtype,))


def _stream_ptr(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need_cuda(name, t, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


@dataclass
class NF4Weight:
    """An NF4-quantized frozen weight [rows, cols] held in device memory."""
    rows: int
    cols: int
    block_size: int
    double_quant: bool
    dq_group: int
    codes: "object"                      # uint8 [rows*cols/2]
    absmax: "object" = None              # float32 [nb]
    absmax_q: "object" = None            # uint8 [nb]
    absmax_scale2: "object" = None       # float32 [ng]

    @property
    def shape(self) -> Tuple[int, int]:
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def size_bytes(self) -> int:
        n = self.codes.numel()
        for t in (self.absmax, self.absmax_q, self.absmax_scale2):
            if t is not None:
                n += t.numel() * t.element_size()
        return n

    def descriptor(self) -> QloraNf4:
        return QloraNf4(self.rows, self.cols, self.block_size, int(self.double_quant),
                        self.dq_group, 0, _ptr(self.codes), _ptr(self.absmax),
                        _ptr(self.absmax_q), _ptr(self.absmax_scale2))


def empty_nf4(rows: int, cols: int, block_size: int = 64, double_quant: bool = False,
              dq_group: int = 256, device="cuda") -> NF4Weight:
    torch = _torch()
    n = rows * cols
    nb = n // block_size if block_size > 0 else 0
    codes = torch.empty(n // 2, dtype=torch.uint8, device=device)
    if double_quant:
        ng = (nb + dq_group - 1) // dq_group
        return NF4Weight(rows, cols, block_size, True, dq_group, codes, None,
                         torch.empty(nb, dtype=torch.uint8, device=device),
                         torch.empty(ng, dtype=torch.float32, device=device))
    return NF4Weight(rows, cols, block_size, False, dq_group, codes,
                     torch.empty(nb, dtype=torch.float32, device=device))


def quantize(w, block_size: int = 64, double_quant: bool = False, dq_group=256) -> NF4Weight:
    """Blockwise NF4 quantization of a 2-D fp32 GPU tensor (optionally with the block
    scales double-quantized to u8 + one fp32 scale per dq_group blocks; dq_group
    "global" puts every block in one group)."""
    torch = _torch()
    _need_cuda("w", w, torch.float32)
    if w.dim() != 2:
        raise ValueError("w must be 2-D [rows, cols]")
    rows, cols = w.shape
    if dq_group == "global":
        dq_group = max(1, (rows * cols) // block_size) if block_size > 0 else 1
    if block_size <= 0 or (rows * cols) % block_size:
        desc_bs = block_size  # let the library produce the status and message
        q = NF4Weight(rows, cols, desc_bs, double_quant, dq_group,
                      torch.empty(0, dtype=torch.uint8, device=w.device))
    else:
        q = empty_nf4(rows, cols, block_size, double_quant, dq_group, w.device)
    d = q.descriptor()
    _lib.check(_lib.lib().qlora_nf4_quantize(_ptr(w), ctypes.byref(d), _stream_ptr(w.device)))
    return q


def dequantize(q: NF4Weight, dtype=None):
    """w_hat = fl32(level * block scale), rounded to nearest-even into ``dtype``."""
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    out = torch.empty(q.rows, q.cols, dtype=dtype, device=q.device)
    d = q.descriptor()
    _lib.check(_lib.lib().qlora_nf4_dequantize(ctypes.byref(d), dtype_code(dtype), _ptr(out),
                                              _stream_ptr(q.device)))
    return out


def workspace_bytes(op: int, m: int, rows: int, cols: int, r: int, dtype, flags: int = 0) -> int:
    return int(_lib.lib().qlora_workspace_bytes(op | (flags << _lib.QLORA_OP_FLAGS_SHIFT), m, rows, cols, r,
                                               dtype_code(dtype)))


_PATHS = {"auto": 0, "fused": _lib.QLORA_FLAG_FUSED, "dequant": _lib.QLORA_FLAG_DEQUANT_GEMM}


def _flags(rslora: bool, path: str) -> int:
    if path not in _PATHS:
        raise ValueError("path must be one of %s" % sorted(_PATHS))
    return (_lib.QLORA_FLAG_RSLORA if rslora else 0) | _PATHS[path]


def _workspace(nbytes: int, device, workspace=None):
    torch = _torch()
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small: %d < %d bytes" % (workspace.numel(), nbytes))
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _flatten(x, cols):
    if x.shape[-1] != cols:
        raise ValueError("last dim of x must be %d, got %d" % (cols, x.shape[-1]))
    lead = tuple(x.shape[:-1])
    return x.reshape(-1, cols), lead


def _dropout_args(dropout_mask, dropout_p, x2):
    torch = _torch()
    if dropout_mask is None:
        return None, 0.0
    mk = dropout_mask.reshape(-1, x2.shape[1]).contiguous()
    _need_cuda("dropout_mask", mk, torch.uint8)
    if mk.shape != x2.shape:
        raise ValueError("dropout_mask must have x's shape")
    return mk, float(dropout_p)


def linear_fwd(q: NF4Weight, x, lora_a, lora_b, alpha: float, bias=None, save_t: bool = False,
               rslora: bool = False, workspace=None, out=None, t_out=None, path: str = "auto",
               dropout_mask=None, dropout_p: float = 0.0):
    """y = x . deq(W)^T + s (x . A^T) . B^T (+ bias), s = alpha / r (alpha / sqrt(r)
    with rslora).  Leading dims of x are flattened to tokens.  Returns y, or
    (y, T0) with T0 = x A^T in fp32 when save_t.  ``out`` / ``t_out`` may supply
    preallocated outputs.  With ``dropout_mask`` (uint8, x's shape, nonzero = kept)
    the low-rank branch reads x * mask / (1 - dropout_p) (LoRA dropout)."""
    torch = _torch()
    dt = x.dtype
    x2, lead = _flatten(x, q.cols)
    x2 = x2.contiguous()
    for name, t in (("x", x2), ("lora_a", lora_a), ("lora_b", lora_b), ("bias", bias)):
        _need_cuda(name, t, dt)
    r = lora_a.shape[0]
    m = x2.shape[0]
    y = out if out is not None else torch.empty(m, q.rows, dtype=dt, device=x.device)
    _need_cuda("out", y, dt)
    if y.numel() != m * q.rows:
        raise ValueError("out must hold %d x %d elements" % (m, q.rows))
    t0 = t_out if t_out is not None else (
        torch.empty(m, r, dtype=torch.float32, device=x.device) if save_t else None)
    _need_cuda("t_out", t0, torch.float32)
    if t0 is not None and t0.numel() != m * r:
        raise ValueError("t_out must hold %d x %d fp32 elements" % (m, r))
    flags = _flags(rslora, path)
    mk, p = _dropout_args(dropout_mask, dropout_p, x2)
    qflags = flags | (_lib.QLORA_FLAG_DROPOUT | _lib.QLORA_FLAG_STORED_MASK if mk is not None else 0)
    ws = _workspace(workspace_bytes(_lib.QLORA_OP_FWD, m, q.rows, q.cols, r, dt, qflags), x.device, workspace)
    d = q.descriptor()
    if mk is None:
        _lib.check(_lib.lib().qlora_linear_fwd(
            ctypes.byref(d), _ptr(x2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), flags,
            _ptr(bias), dtype_code(dt), _ptr(y), _ptr(t0), _ptr(ws), ws.numel() * ws.element_size(),
            _stream_ptr(x.device)))
    else:
        _lib.check(_lib.lib().qlora_linear_fwd_dropout(
            ctypes.byref(d), _ptr(x2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), flags,
            _ptr(bias), dtype_code(dt), _ptr(mk), p, _ptr(y), _ptr(t0), _ptr(ws), ws.numel() * ws.element_size(),
            _stream_ptr(x.device)))
    y = y.reshape(*lead, q.rows)
    return (y, t0) if (save_t or t_out is not None) else y


def linear_fwd_noalloc(q: NF4Weight, x, lora_a, lora_b, alpha: float, bias=None, out=None, t_out=None,
                       rslora: bool = False, path: str = "auto"):
    """The forward through qlora_linear_fwd_noalloc: no workspace, the library's own
    scratch array instead (for graph capture and serving loops that cannot
    allocate).  ``out`` (and ``t_out`` for T0) may be preallocated; returns y, or
    (y, T0) when ``t_out`` is given."""
    torch = _torch()
    dt = x.dtype
    x2, lead = _flatten(x, q.cols)
    x2 = x2.contiguous()
    for name, t in (("x", x2), ("lora_a", lora_a), ("lora_b", lora_b), ("bias", bias)):
        _need_cuda(name, t, dt)
    r = lora_a.shape[0]
    m = x2.shape[0]
    y = out if out is not None else torch.empty(m, q.rows, dtype=dt, device=x.device)
    _need_cuda("out", y, dt)
    _need_cuda("t_out", t_out, torch.float32)
    if y.numel() != m * q.rows or (t_out is not None and t_out.numel() != m * r):
        raise ValueError("out / t_out have the wrong size")
    d = q.descriptor()
    _lib.check(_lib.lib().qlora_linear_fwd_noalloc(
        ctypes.byref(d), _ptr(x2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), _flags(rslora, path),
        _ptr(bias), dtype_code(dt), _ptr(y), _ptr(t_out), _stream_ptr(x.device)))
    y = y.reshape(*lead, q.rows)
    return (y, t_out) if t_out is not None else y


def linear_fwd_cached(w_cd, x, lora_a, lora_b, alpha: float, bias=None, save_t: bool = False,
                      rslora: bool = False, workspace=None, out=None, t_out=None):
    """Cached-dequant forward: ``w_cd`` is W~ [rows, cols] in x's dtype (bf16 / f16),
    dequantized once by ``dequantize(q, dtype)`` and kept by the caller; returns
    x . w_cd^T + s (x . A^T) . B^T (+ bias), or (y, T0) when save_t."""
    torch = _torch()
    dt = x.dtype
    rows, cols = w_cd.shape
    _need_cuda("w_cd", w_cd, dt)
    x2, lead = _flatten(x, cols)
    x2 = x2.contiguous()
    for name, t in (("x", x2), ("lora_a", lora_a), ("lora_b", lora_b), ("bias", bias)):
        _need_cuda(name, t, dt)
    r = lora_a.shape[0]
    m = x2.shape[0]
    y = out if out is not None else torch.empty(m, rows, dtype=dt, device=x.device)
    _need_cuda("out", y, dt)
    if y.numel() != m * rows:
        raise ValueError("out must hold %d x %d elements" % (m, rows))
    t0 = t_out if t_out is not None else (
        torch.empty(m, r, dtype=torch.float32, device=x.device) if save_t else None)
    _need_cuda("t_out", t0, torch.float32)
    if t0 is not None and t0.numel() != m * r:
        raise ValueError("t_out must hold %d x %d fp32 elements" % (m, r))
    flags = _lib.QLORA_FLAG_RSLORA if rslora else 0
    ws = _workspace(workspace_bytes(_lib.QLORA_OP_FWD_CACHED, m, rows, cols, r, dt, flags), x.device, workspace)
    _lib.check(_lib.lib().qlora_linear_fwd_cached(
        _ptr(w_cd.contiguous()), rows, cols, _ptr(x2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), flags,
        _ptr(bias), dtype_code(dt), _ptr(y), _ptr(t0), _ptr(ws), ws.numel() * ws.element_size(),
        _stream_ptr(x.device)))
    y = y.reshape(*lead, rows)
    return (y, t0) if (save_t or t_out is not None) else y


class _GroupArgs:
    """ctypes arrays for the g projections of a group call (kept alive with it)."""

    def __init__(self, qs, lora_as=None, lora_bs=None, alphas=None):
        g = len(qs)
        if not 1 <= g <= _lib.QLORA_GROUP_MAX:
            raise ValueError("a group holds 1 to %d projections" % _lib.QLORA_GROUP_MAX)
        self.g = g
        self.descs = [q.descriptor() for q in qs]
        self.w = (ctypes.POINTER(_lib.QloraNf4) * g)(*[ctypes.pointer(d) for d in self.descs])
        ranks = [a.shape[0] for a in lora_as] if lora_as is not None else [0] * g
        self.r = (ctypes.c_int32 * g)(*ranks)
        if lora_as is not None:
            self.a = (ctypes.c_void_p * g)(*[_ptr(a) for a in lora_as])
            self.b = (ctypes.c_void_p * g)(*[_ptr(b) for b in lora_bs])
            self.alpha = (ctypes.c_float * g)(*[float(a) for a in alphas])

    @staticmethod
    def ptrs(ts):
        return None if ts is None else (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])


def group_workspace_bytes(op: int, qs, m: int, ranks, dtype) -> int:
    """Workspace bytes of a group call (op QLORA_OP_FWD / QLORA_OP_BWD)."""
    ga = _GroupArgs(qs)
    ga.r = (ctypes.c_int32 * ga.g)(*[int(r) for r in ranks])
    return int(_lib.lib().qlora_group_workspace_bytes(op, ga.g, ga.w, m, ga.r, dtype_code(dtype)))


def linear_fwd_group(qs, x, lora_as, lora_bs, alphas, bias=None, save_t: bool = False, rslora: bool = False,
                     workspace=None, out=None):
    """Projections that read the same x in one call: returns y [m, sum rows_i] with
    projection i's output in its columns (and the list of T0_i = x A_i^T in fp32 when
    save_t).  bias, if given, is [sum rows_i]."""
    torch = _torch()
    dt = x.dtype
    cols = qs[0].cols
    x2, lead = _flatten(x, cols)
    x2 = x2.contiguous()
    _need_cuda("x", x2, dt)
    for i, (a, b) in enumerate(zip(lora_as, lora_bs)):
        _need_cuda("lora_a[%d]" % i, a, dt)
        _need_cuda("lora_b[%d]" % i, b, dt)
    _need_cuda("bias", bias, dt)
    m = x2.shape[0]
    N = sum(q.rows for q in qs)
    y = out if out is not None else torch.empty(m, N, dtype=dt, device=x.device)
    _need_cuda("out", y, dt)
    if y.numel() != m * N:
        raise ValueError("out must hold %d x %d elements" % (m, N))
    ts = [torch.empty(m, a.shape[0], dtype=torch.float32, device=x.device) for a in lora_as] if save_t else None
    ga = _GroupArgs(qs, lora_as, lora_bs, alphas)
    ws = _workspace(group_workspace_bytes(_lib.QLORA_OP_FWD, qs, m, [a.shape[0] for a in lora_as], dt), x.device,
                    workspace)
    _lib.check(_lib.lib().qlora_linear_fwd_group(
        ga.g, ga.w, _ptr(x2), m, ga.a, ga.b, ga.r, ga.alpha, _lib.QLORA_FLAG_RSLORA if rslora else 0, _ptr(bias),
        dtype_code(dt), _ptr(y), _GroupArgs.ptrs(ts), _ptr(ws), ws.numel() * ws.element_size(),
        _stream_ptr(x.device)))
    y = y.reshape(*lead, N)
    return (y, ts) if save_t else y


def linear_bwd_group(qs, x, dy, lora_as, lora_bs, alphas, t_saved=None, need_dx: bool = True,
                     rslora: bool = False, workspace=None):
    """Gradients of a group with the bases frozen: dy [m, sum rows_i] laid out like the
    forward's y.  Returns (dX = sum of the projections' input gradients, or None;
    the list of dA_i fp32; the list of dB_i fp32)."""
    torch = _torch()
    dt = x.dtype
    cols = qs[0].cols
    N = sum(q.rows for q in qs)
    x2, lead = _flatten(x, cols)
    dy2, _ = _flatten(dy, N)
    x2, dy2 = x2.contiguous(), dy2.contiguous()
    _need_cuda("x", x2, dt)
    _need_cuda("dy", dy2, dt)
    m = x2.shape[0]
    dx = torch.empty(m, cols, dtype=dt, device=x.device) if need_dx else None
    das = [torch.empty(a.shape[0], cols, dtype=torch.float32, device=x.device) for a in lora_as]
    dbs = [torch.empty(q.rows, a.shape[0], dtype=torch.float32, device=x.device) for q, a in zip(qs, lora_as)]
    if t_saved is not None:
        for t in t_saved:
            _need_cuda("t_saved", t, torch.float32)
    ga = _GroupArgs(qs, lora_as, lora_bs, alphas)
    ws = _workspace(group_workspace_bytes(_lib.QLORA_OP_BWD, qs, m, [a.shape[0] for a in lora_as], dt), x.device,
                    workspace)
    _lib.check(_lib.lib().qlora_linear_bwd_group(
        ga.g, ga.w, _ptr(x2), _ptr(dy2), m, ga.a, ga.b, ga.r, ga.alpha, _lib.QLORA_FLAG_RSLORA if rslora else 0,
        dtype_code(dt), _GroupArgs.ptrs(t_saved), _ptr(dx), _GroupArgs.ptrs(das), _GroupArgs.ptrs(dbs), _ptr(ws),
        ws.numel() * ws.element_size(), _stream_ptr(x.device)))
    if dx is not None:
        dx = dx.reshape(*lead, cols)
    return dx, das, dbs


def linear_bwd(q: NF4Weight, x, dy, lora_a, lora_b, alpha: float, t_saved=None, need_dx: bool = True,
               rslora: bool = False, workspace=None, dx_out=None, da_out=None, db_out=None, path: str = "auto",
               dropout_mask=None, dropout_p: float = 0.0):
    """Gradients with the base frozen: returns (dX or None, dA fp32 [r, cols], dB fp32 [rows, r]).
    ``*_out`` may supply preallocated outputs; ``dropout_mask`` / ``dropout_p`` as in
    the forward (the same mask)."""
    torch = _torch()
    dt = x.dtype
    x2, lead = _flatten(x, q.cols)
    dy2, _ = _flatten(dy, q.rows)
    x2, dy2 = x2.contiguous(), dy2.contiguous()
    for name, t in (("x", x2), ("dy", dy2), ("lora_a", lora_a), ("lora_b", lora_b)):
        _need_cuda(name, t, dt)
    _need_cuda("t_saved", t_saved, torch.float32)
    r = lora_a.shape[0]
    m = x2.shape[0]
    dx = dx_out if dx_out is not None else (
        torch.empty(m, q.cols, dtype=dt, device=x.device) if need_dx else None)
    da = da_out if da_out is not None else torch.empty(r, q.cols, dtype=torch.float32, device=x.device)
    db = db_out if db_out is not None else torch.empty(q.rows, r, dtype=torch.float32, device=x.device)
    _need_cuda("dx_out", dx, dt)
    _need_cuda("da_out", da, torch.float32)
    _need_cuda("db_out", db, torch.float32)
    if (dx is not None and dx.numel() != m * q.cols) or da.numel() != r * q.cols or db.numel() != q.rows * r:
        raise ValueError("output buffers have the wrong size")
    if t_saved is not None and t_saved.numel() != m * r:
        raise ValueError("t_saved must hold %d x %d fp32 elements" % (m, r))
    flags = _flags(rslora, path)
    mk, p = _dropout_args(dropout_mask, dropout_p, x2)
    qflags = flags | (_lib.QLORA_FLAG_DROPOUT | _lib.QLORA_FLAG_STORED_MASK if mk is not None else 0)
    ws = _workspace(workspace_bytes(_lib.QLORA_OP_BWD, m, q.rows, q.cols, r, dt, qflags), x.device, workspace)
    d = q.descriptor()
    if mk is None:
        _lib.check(_lib.lib().qlora_linear_bwd(
            ctypes.byref(d), _ptr(x2), _ptr(dy2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), flags,
            dtype_code(dt), _ptr(t_saved), _ptr(dx), _ptr(da), _ptr(db), _ptr(ws),
            ws.numel() * ws.element_size(), _stream_ptr(x.device)))
    else:
        _lib.check(_lib.lib().qlora_linear_bwd_dropout(
            ctypes.byref(d), _ptr(x2), _ptr(dy2), m, _ptr(lora_a), _ptr(lora_b), r, float(alpha), flags,
            dtype_code(dt), _ptr(mk), p, _ptr(t_saved), _ptr(dx), _ptr(da), _ptr(db), _ptr(ws),
            ws.numel() * ws.element_size(), _stream_ptr(x.device)))
    if dx is not None:
        dx = dx.reshape(*lead, q.cols)
    return dx, da, db


def _check_like(name, t, device, dtype, shape):
    """A contiguous ``dtype`` tensor of ``shape`` on ``device``."""
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be a GPU tensor on %s" % (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous and of shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _check_adapter(q, lora_a, lora_b, device, dtype, at=""):
    if q.device != device:
        raise ValueError("the weight%s is on %s, x on %s" % (at, q.device, device))
    if lora_a.dim() != 2:
        raise ValueError("lora_a%s must be [r, %d]" % (at, q.cols))
    r = lora_a.shape[0]
    _check_like("lora_a" + at, lora_a, device, dtype, (r, q.cols))
    _check_like("lora_b" + at, lora_b, device, dtype, (q.rows, r))
    return r


def _grad_code(grad_dtype, dtype):
    torch = _torch()
    grad_dtype = torch.float32 if grad_dtype is None else grad_dtype
    if grad_dtype not in (torch.float32, dtype):
        raise TypeError("grad_dtype must be torch.float32 or %s, got %s" % (dtype, grad_dtype))
    return grad_dtype, dtype_code(grad_dtype)


def _dropout_call(q, x, lora_a, lora_b, p, seed, rslora, path):
    """What the two seeded dropout calls share: (x as tokens, lead, rank, flags)."""
    torch = _torch()
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    dtype_code(x.dtype)
    x2, lead = _flatten(x, q.cols)
    r = _check_adapter(q, lora_a, lora_b, x.device, x.dtype)
    _check_like("seed", seed, x.device, torch.int64, (2,))
    if not 0.0 <= p < 1.0:
        raise ValueError("p must lie in [0, 1), got %r" % (p,))
    return x2.contiguous(), lead, r, _flags(rslora, path)


def linear_fwd_dropout(q: NF4Weight, x, lora_a, lora_b, alpha: float, p: float, seed, bias=None, save_t: bool = False,
                       rslora: bool = False, workspace=None, out=None, path: str = "auto"):
    """``linear_fwd`` with LoRA dropout whose mask is drawn on the fly and never stored: the
    low-rank branch reads x * M / (1 - p), M[i, k] from Philox 4x32-10 under ``seed``, an int64
    GPU tensor [2] = (seed, offset) that is read on the device (a captured call draws anew at each
    replay that finds other values there).  p counts in 65536ths (rounded to the nearest, at most
    65535).  Returns y, or (y, T0) with T0 = (x M) A^T in fp32 when save_t; the backward takes
    the same seed and offset."""
    torch = _torch()
    x2, lead, r, flags = _dropout_call(q, x, lora_a, lora_b, p, seed, rslora, path)
    dt, m = x2.dtype, x2.shape[0]
    if bias is not None:
        _check_tensor("bias", bias, x.device, dt, q.rows)
    if out is None:
        y = torch.empty(m, q.rows, dtype=dt, device=x.device)
    else:
        _check_tensor("out", out, x.device, dt, m * q.rows)
        y = out
    t0 = torch.empty(m, r, dtype=torch.float32, device=x.device) if save_t else None
    if m:
        ws = _workspace_on(x.device, workspace_bytes(_lib.QLORA_OP_FWD, m, q.rows, q.cols, r, dt,
                                                     flags | _lib.QLORA_FLAG_DROPOUT), workspace)
        d = q.descriptor()
        _launch(x.device, _lib.lib().qlora_linear_fwd_dropout_seeded, ctypes.byref(d), _ptr(x2), m, _ptr(lora_a),
                _ptr(lora_b), r, float(alpha), flags, _ptr(bias), dtype_code(dt), _ptr(seed), float(p), _ptr(y), _ptr(t0),
                _ptr(ws), ws.numel() * ws.element_size())
    y = y.view(*lead, q.rows)
    return (y, t0) if save_t else y


def linear_bwd_dropout(q: NF4Weight, x, dy, lora_a, lora_b, alpha: float, p: float, seed, t_saved=None,
                       need_dx: bool = True, rslora: bool = False, grad_dtype=None, workspace=None, path: str = "auto"):
    """Gradients of ``linear_fwd_dropout`` with the base frozen, under the forward's p and seed:
    (dX or None, dA [r, cols], dB [rows, r]); ``t_saved`` is the forward's T0 (else recomputed).
    ``grad_dtype``: torch.float32 (the default, what ``adamw_step`` takes) or x's dtype."""
    torch = _torch()
    x2, lead, r, flags = _dropout_call(q, x, lora_a, lora_b, p, seed, rslora, path)
    dt, m = x2.dtype, x2.shape[0]
    dy2 = _flatten(dy, q.rows)[0].contiguous()
    _check_like("dy", dy2, x.device, dt, (m, q.rows))
    if t_saved is not None:
        _check_like("t_saved", t_saved, x.device, torch.float32, (m, r))
    gt, gd = _grad_code(grad_dtype, dt)
    dx = torch.empty(m, q.cols, dtype=dt, device=x.device) if need_dx else None
    da = torch.empty(r, q.cols, dtype=gt, device=x.device)
    db = torch.empty(q.rows, r, dtype=gt, device=x.device)
    ws = _workspace_on(x.device, workspace_bytes(_lib.QLORA_OP_BWD, m, q.rows, q.cols, r, dt,
                                                 flags | _lib.QLORA_FLAG_DROPOUT), workspace)
    d = q.descriptor()
    _launch(x.device, _lib.lib().qlora_linear_bwd_dropout_seeded, ctypes.byref(d), _ptr(x2), _ptr(dy2), m, _ptr(lora_a),
            _ptr(lora_b), r, float(alpha), flags, dtype_code(dt), _ptr(seed), float(p), _ptr(t_saved), gd, _ptr(dx),
            _ptr(da), _ptr(db), _ptr(ws), ws.numel() * ws.element_size())
    return (None if dx is None else dx.view(*lead, q.cols)), da, db


def gated_workspace_bytes(op: int, qs, m: int, ranks, dtype) -> int:
    """Workspace bytes of linear_fwd_gated (op QLORA_OP_FWD) or linear_bwd_gated (QLORA_OP_BWD)."""
    ga = _GroupArgs(qs)
    ga.r = (ctypes.c_int32 * ga.g)(*[int(r) for r in ranks])
    return int(_lib.lib().qlora_gated_workspace_bytes(op, ga.w, m, ga.r, dtype_code(dtype)))


_Two = ctypes.c_void_p * 2
_TwoInts = ctypes.c_int32 * 2
_TwoFloats = ctypes.c_float * 2
_TwoWeights = _lib.QloraNf4 * 2


def _two(ts):
    return None if ts is None else _Two(_ptr(ts[0]), _ptr(ts[1]))


class _GatedArgs:
    """ctypes arrays of a gated block's two projections (kept alive with it)."""

    __slots__ = ("descs", "w", "r", "a", "b", "alpha")

    def __init__(self, qs, ranks, lora_as, lora_bs, alphas):
        self.descs = _TwoWeights(qs[0].descriptor(), qs[1].descriptor())
        at = ctypes.addressof(self.descs)
        self.w = _Two(at, at + ctypes.sizeof(_lib.QloraNf4))
        self.r = _TwoInts(*ranks)
        self.a = _two(lora_as)
        self.b = _two(lora_bs)
        self.alpha = _TwoFloats(float(alphas[0]), float(alphas[1]))


def _gated_call(qs, x, lora_as, lora_bs, alphas, act):
    if len(qs) != 2 or len(lora_as) != 2 or len(lora_bs) != 2 or len(alphas) != 2:
        raise ValueError("a gated block takes two projections (gate, up) with an adapter and an alpha each")
    if act not in _lib.QLORA_ACTS:
        raise ValueError("act must be one of %s, got %r" % (sorted(_lib.QLORA_ACTS), act))
    if qs[0].rows != qs[1].rows or qs[0].cols != qs[1].cols:
        raise ValueError("gate is [%d, %d], up [%d, %d]" % (qs[0].rows, qs[0].cols, qs[1].rows, qs[1].cols))
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    dtype_code(x.dtype)
    x2, lead = _flatten(x, qs[0].cols)
    ranks = [_check_adapter(q, a, b, x.device, x.dtype, "[%d]" % i)
             for i, (q, a, b) in enumerate(zip(qs, lora_as, lora_bs))]
    return x2.contiguous(), lead, ranks, _GatedArgs(qs, ranks, lora_as, lora_bs, alphas)


def linear_fwd_gated(qs, x, lora_as, lora_bs, alphas, act: str = "silu", bias=None, save: bool = False,
                     rslora: bool = False, workspace=None, out=None):
    """The gated feed-forward block over two projections of the same x, qs = (gate, up):
    h [m, rows] = act(g) u with g and u as ``linear_fwd`` gives them; act "silu", "gelu" or
    "gelu_tanh"; bias, if given, is [2 rows] (gate, then up).  With ``save`` returns (h, pre, ts)
    for the backward: pre [m, 2 rows] = [g | u] in x's dtype, ts the T0_i = x A_i^T in fp32."""
    torch = _torch()
    x2, lead, ranks, ga = _gated_call(qs, x, lora_as, lora_bs, alphas, act)
    dt, m, rows, device = x2.dtype, x2.shape[0], qs[0].rows, x.device
    if bias is not None:
        _check_tensor("bias", bias, device, dt, 2 * rows)
    if out is None:
        h = torch.empty(m, rows, dtype=dt, device=device)
    else:
        _check_tensor("out", out, device, dt, m * rows)
        h = out
    pre = torch.empty(m, 2 * rows, dtype=dt, device=device) if save else None
    ts = [torch.empty(m, r, dtype=torch.float32, device=device) for r in ranks] if save else None
    if m:
        lib, code = _lib.lib(), dtype_code(dt)
        ws = _workspace_on(device, int(lib.qlora_gated_workspace_bytes(_lib.QLORA_OP_FWD, ga.w, m, ga.r, code)), workspace)
        _launch(device, lib.qlora_linear_fwd_gated, ga.w, _ptr(x2), m, ga.a, ga.b, ga.r, ga.alpha,
                _lib.QLORA_FLAG_RSLORA if rslora else 0, _lib.QLORA_ACTS[act], _ptr(bias), code, _ptr(h), _ptr(pre),
                _two(ts), _ptr(ws), ws.numel() * ws.element_size())
    h = h.view(*lead, rows)
    return (h, pre, ts) if save else h


def linear_bwd_gated(qs, x, dh, lora_as, lora_bs, alphas, pre, act: str = "silu", t_saved=None, need_dx: bool = True,
                     rslora: bool = False, grad_dtype=None, workspace=None):
    """Gradients of ``linear_fwd_gated`` with the bases frozen, from dh [m, rows] and the ``pre``
    it saved: (dX or None, [dA_gate, dA_up], [dB_gate, dB_up]).  ``t_saved``: its ts (else
    recomputed).  ``grad_dtype``: the adapters' gradients in torch.float32 (the default, what
    ``adamw_step`` takes) or x's dtype."""
    torch = _torch()
    x2, lead, ranks, ga = _gated_call(qs, x, lora_as, lora_bs, alphas, act)
    dt, m, rows, cols, device = x2.dtype, x2.shape[0], qs[0].rows, qs[0].cols, x.device
    dh2 = _flatten(dh, rows)[0].contiguous()
    _check_like("dh", dh2, device, dt, (m, rows))
    _check_tensor("pre", pre, device, dt, m * 2 * rows)
    if t_saved is not None:
        if len(t_saved) != 2:
            raise ValueError("t_saved must hold two tensors")
        for i, (t, r) in enumerate(zip(t_saved, ranks)):
            _check_like("t_saved[%d]" % i, t, device, torch.float32, (m, r))
    gt, gd = _grad_code(grad_dtype, dt)
    dx = torch.empty(m, cols, dtype=dt, device=device) if need_dx else None
    das = [torch.empty(r, cols, dtype=gt, device=device) for r in ranks]
    dbs = [torch.empty(rows, r, dtype=gt, device=device) for r in ranks]
    lib, code = _lib.lib(), dtype_code(dt)
    ws = _workspace_on(device, int(lib.qlora_gated_workspace_bytes(_lib.QLORA_OP_BWD, ga.w, m, ga.r, code)), workspace)
    _launch(device, lib.qlora_linear_bwd_gated, ga.w, _ptr(x2), _ptr(dh2), _ptr(pre), m, ga.a, ga.b, ga.r, ga.alpha,
            _lib.QLORA_FLAG_RSLORA if rslora else 0, _lib.QLORA_ACTS[act], code, _two(t_saved), gd, _ptr(dx),
            _two(das), _two(dbs), _ptr(ws), ws.numel() * ws.element_size())
    return (None if dx is None else dx.view(*lead, cols)), das, dbs


def merge(q: NF4Weight, lora_a, lora_b, alpha: float, rslora: bool = False, out=None):
    """Dense merged weight RNE(w_hat + s B A) [rows, cols] in the adapters' dtype
    (never re-quantized to NF4).  ``out`` may supply a preallocated output."""
    torch = _torch()
    dt = lora_a.dtype
    _need_cuda("lora_a", lora_a, dt)
    _need_cuda("lora_b", lora_b, dt)
    r = lora_a.shape[0]
    if lora_a.dim() != 2 or lora_a.shape[1] != q.cols:
        raise ValueError("lora_a must be [r, %d]" % q.cols)
    if lora_b.dim() != 2 or tuple(lora_b.shape) != (q.rows, r):
        raise ValueError("lora_b must be [%d, %d]" % (q.rows, r))
    o = out if out is not None else torch.empty(q.rows, q.cols, dtype=dt, device=lora_a.device)
    _need_cuda("out", o, dt)
    if o.numel() != q.rows * q.cols:
        raise ValueError("out must hold %d x %d elements" % (q.rows, q.cols))
    d = q.descriptor()
    _lib.check(_lib.lib().qlora_merge(ctypes.byref(d), _ptr(lora_a), _ptr(lora_b), r, float(alpha),
                                      _lib.QLORA_FLAG_RSLORA if rslora else 0, dtype_code(dt), _ptr(o),
                                      _stream_ptr(lora_a.device)))
    return o.view(q.rows, q.cols)


def mse_loss_grad(y, target, dy=None):
    """loss = mean((y - target)^2) (a 1-element fp32 GPU tensor) and dy = 2 (y - target) / n
    in y's dtype."""
    torch = _torch()
    dt = y.dtype
    _need_cuda("y", y, dt)
    _need_cuda("target", target, dt)
    if y.numel() != target.numel():
        raise ValueError("y and target differ in size")
    dy = dy if dy is not None else torch.empty_like(y)
    _need_cuda("dy", dy, dt)
    loss = torch.empty(1, dtype=torch.float32, device=y.device)
    ws = torch.empty(_lib.QLORA_MSE_WORKSPACE_BYTES, dtype=torch.uint8, device=y.device)
    _lib.check(_lib.lib().qlora_mse_loss_grad(_ptr(y), _ptr(target), y.numel(), dtype_code(dt), _ptr(loss),
                                              _ptr(dy), _ptr(ws), ws.numel(), _stream_ptr(y.device)))
    return loss, dy


def _launch(device, call, *args):
    """call(*args, stream) with ``device`` current (its current stream); raises on an error."""
    cuda, index = _torch()._C, device.index
    if index == cuda._cuda_getDevice():
        _lib.check(call(*args, cuda._cuda_getCurrentRawStream(index)))
    else:
        with _torch().cuda.device(device):
            _lib.check(call(*args, cuda._cuda_getCurrentRawStream(index)))


def _check_tensor(name, t, device, dtype, numel):
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.numel() != numel:
        raise ValueError("%s must hold %d elements, got %d" % (name, numel, t.numel()))


def _workspace_on(device, nbytes, workspace):
    torch = _torch()
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not workspace.is_cuda or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % (device,))
    return _workspace(nbytes, device, workspace)


def _strided_rows(x, cols):
    """x as rows of ``cols`` contiguous elements and the stride between them (a view where
    the layout allows, else a copy), with the leading dims (None: x is 2-D already)."""
    if x.shape[-1] != cols:
        raise ValueError("last dim must be %d, got %d" % (cols, x.shape[-1]))
    lead = None
    if x.dim() != 2:
        lead = tuple(x.shape[:-1])
        x = x.reshape(-1, cols)
    if x.is_contiguous():
        return x, cols, lead
    if x.shape[0] <= 1:
        return (x if x.stride(1) == 1 else x.contiguous()), cols, lead
    if (cols > 1 and x.stride(1) != 1) or x.stride(0) < cols:
        return x.contiguous(), cols, lead
    return x, x.stride(0), lead


@dataclass
class Int8Weight:
    """A weight [rows, cols] (or one for each expert, [experts, rows, cols]) in 8 bits with a
    scale per output channel, held in device memory."""
    rows: int
    cols: int
    codes: "object"        # int8 [experts, rows, ld], ld = cols rounded up to 128, zeros past cols
    scale: "object"        # float32 [experts, rows]

    @property
    def experts(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self) -> Tuple[int, ...]:
        return (self.rows, self.cols) if self.experts == 1 else (self.experts, self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def size_bytes(self) -> int:
        return self.codes.numel() + 4 * self.scale.numel()

    def __getstate__(self):  # the descriptor holds addresses: a copy makes its own
        return {k: v for k, v in self.__dict__.items() if k != "_made"}

    def descriptor(self) -> QloraInt8:
        return self._described()[0]

    def _described(self):
        """The descriptor, and (rows, cols, experts)."""
        # Kept between calls as long as all it was made from is the same: the tensors' storages
        # can be replaced under them (``codes.data = ...``), and the fields assigned.
        c, s = self.codes, self.scale
        key = (self.rows, self.cols, c.data_ptr(), s.data_ptr(), c.shape, s.shape, c.dtype, s.dtype, c.is_contiguous(),
               s.is_contiguous())
        made = self.__dict__.get("_made")
        if made is None or made[0] != key:
            torch = _torch()
            ld = (self.cols + 127) // 128 * 128
            for name, t, dt, shape in (("codes", c, torch.int8, (self.experts, self.rows, ld)),
                                       ("scale", s, torch.float32, (self.experts, self.rows))):
                if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda or \
                        t.device != c.device:
                    raise ValueError("%s must be a contiguous %s GPU tensor of shape %s" % (name, dt, shape))
            shape = (self.rows, self.cols, self.experts)
            made = self.__dict__["_made"] = (key, (QloraInt8(*shape, 0, _ptr(c), _ptr(s)), shape))
        return made[1]


def quantize_int8(w) -> Int8Weight:
    """8-bit codes and one scale per row of a [rows, cols] weight (fp32, bf16 or f16; for
    instance the dense result of ``merge``), or of one weight per expert
    [experts, rows, cols].  Rows may be strided."""
    torch = _torch()
    if not w.is_cuda:
        raise ValueError("w must be a GPU tensor")
    if w.dim() not in (2, 3) or (w.dim() == 3 and w.shape[0] < 1):
        raise ValueError("w must be [rows, cols] or [experts, rows, cols] with at least one expert")
    experts = w.shape[0] if w.dim() == 3 else 1
    rows, cols = w.shape[-2], w.shape[-1]
    if cols > _lib.QLORA_INT8_MAX_COLS:  # before anything is allocated
        raise QloraError(-4, "int8_quantize: %d cols (at most %d)" % (cols, _lib.QLORA_INT8_MAX_COLS))
    ld = (cols + 127) // 128 * 128
    q = Int8Weight(rows, cols, torch.empty(experts, rows, ld, dtype=torch.int8, device=w.device),
                   torch.empty(experts, rows, dtype=torch.float32, device=w.device))
    if rows == 0 or cols == 0:
        return q
    w2, ldw, _ = _strided_rows(w, cols)
    d = q.descriptor()
    _launch(w.device, _lib.lib().qlora_int8_quantize, _ptr(w2), ldw, dtype_code(w.dtype), ctypes.byref(d))
    return q


def int8_workspace_bytes(w: Int8Weight, m: int, grouped: bool = False) -> int:
    """Workspace bytes of linear_int8 (or, grouped, of linear_int8_experts) on m tokens."""
    d = w.descriptor()
    return int(_lib.lib().qlora_int8_workspace_bytes(ctypes.byref(d), m, int(grouped)))


@functools.lru_cache(maxsize=4096)
def _int8_bytes(shape, m, grouped):
    """The same from the weight's rows, cols and experts alone."""
    d = QloraInt8(*shape, 0, None, None)
    return int(_lib.lib().qlora_int8_workspace_bytes(ctypes.byref(d), m, grouped))


def _int8_call(w, x, offsets, bias, out, workspace):
    torch = _torch()
    dt, device = x.dtype, x.device
    code = dtype_code(dt)
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if w.codes.device != device:
        raise ValueError("w is on %s, x on %s" % (w.codes.device, device))
    x2, ldx, lead = _strided_rows(x, w.cols)
    m = x2.shape[0]
    if out is None:
        y = torch.empty(m, w.rows, dtype=dt, device=device)
    else:
        _check_tensor("out", out, device, dt, m * w.rows)
        y = out
    grouped = offsets is not None
    if bias is not None:
        _check_tensor("bias", bias, device, dt, w.rows * (w.experts if grouped else 1))
    d, shape = w._described()
    lib = _lib.lib()
    ws = _workspace_on(device, _int8_bytes(shape, m, grouped), workspace)
    d = ctypes.byref(d)
    ws_bytes = ws.numel() * ws.element_size()
    if grouped:
        _launch(device, lib.qlora_int8_linear_experts, d, x2.data_ptr(), m, ldx, offsets.data_ptr(), _ptr(bias), code,
                y.data_ptr(), ws.data_ptr(), ws_bytes)
    else:
        _launch(device, lib.qlora_int8_linear, d, x2.data_ptr(), m, ldx, _ptr(bias), code, y.data_ptr(),
                ws.data_ptr(), ws_bytes)
    if lead is None and y.dim() == 2:
        return y if y.shape[1] == w.rows else y.view(m, w.rows)
    return y.view(*((m,) if lead is None else lead), w.rows)


def linear_int8(w: Int8Weight, x, bias=None, out=None, workspace=None):
    """y = x . W^T (+ bias) in 8-bit integers: each row of x gets a scale of its own and is
    brought to 8 bits within the call, the sums are exact, y has x's dtype.  Leading dims of
    x are flattened to tokens; rows of x may be strided.  ``out`` may supply a preallocated
    output, which must not overlap x."""
    if w.experts != 1:
        raise ValueError("w holds %d experts: linear_int8_experts takes those" % w.experts)
    return _int8_call(w, x, None, bias, out, workspace)


def linear_int8_experts(w: Int8Weight, x, offsets, bias=None, out=None, workspace=None):
    """The same for rows sorted by expert: rows offsets[e] .. offsets[e + 1] - 1 of x take
    expert e's weight (and bias[e]).  ``offsets``: int32 GPU tensor [experts + 1], read on the
    device.  Rows that no expert has are left as they were in ``out`` (and are unspecified
    without ``out``)."""
    _check_tensor("offsets", offsets, x.device, _torch().int32, w.experts + 1)
    return _int8_call(w, x, offsets, bias, out, workspace)


@dataclass
class Fp8Weight:
    """A weight [rows, cols] in 8-bit floats (e4m3) with a power-of-two scale for each block of
    128 x 128, held in device memory."""
    rows: int
    cols: int
    codes: "object"        # uint8 [rows, ld], ld = cols rounded up to 128, zeros past cols
    scale: "object"        # uint8 [ceil(rows / 128), ceil(cols / 512) * 4]: exponents + 127

    @property
    def shape(self) -> Tuple[int, ...]:
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def size_bytes(self) -> int:
        return self.codes.numel() + self.scale.numel()

    def __getstate__(self):  # the descriptor holds addresses: a copy makes its own
        return {k: v for k, v in self.__dict__.items() if k != "_made"}

    def descriptor(self) -> QloraFp8:
        # Kept between calls as long as all it was made from is the same (as Int8Weight's).
        c, s = self.codes, self.scale
        key = (self.rows, self.cols, c.data_ptr(), s.data_ptr(), c.shape, s.shape, c.dtype, s.dtype, c.is_contiguous(),
               s.is_contiguous())
        made = self.__dict__.get("_made")
        if made is None or made[0] != key:
            torch = _torch()
            for name, t, shape in (("codes", c, _fp8_shapes(self.rows, self.cols)[0]),
                                   ("scale", s, _fp8_shapes(self.rows, self.cols)[1])):
                if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda or \
                        t.device != c.device:
                    raise ValueError("%s must be a contiguous uint8 GPU tensor of shape %s" % (name, shape))
            made = self.__dict__["_made"] = (key, QloraFp8(self.rows, self.cols, 0, _ptr(c), _ptr(s)))
        return made[1]


def _fp8_shapes(rows, cols):
    return (rows, (cols + 127) // 128 * 128), ((rows + 127) // 128, (cols + 511) // 512 * 4)


def quantize_fp8(w) -> Fp8Weight:
    """8-bit floats and one power-of-two scale per block of 128 x 128 of a [rows, cols] weight
    (fp32, bf16 or f16; for instance the dense result of ``merge``).  Rows may be strided."""
    torch = _torch()
    if not w.is_cuda:
        raise ValueError("w must be a GPU tensor")
    if w.dim() != 2:
        raise ValueError("w must be [rows, cols]")
    rows, cols = w.shape
    if cols > _lib.QLORA_FP8_MAX_COLS:  # before anything is allocated
        raise QloraError(-4, "fp8_quantize: %d cols (at most %d)" % (cols, _lib.QLORA_FP8_MAX_COLS))
    code = dtype_code(w.dtype)
    shapes = _fp8_shapes(rows, cols)
    q = Fp8Weight(rows, cols, torch.empty(shapes[0], dtype=torch.uint8, device=w.device),
                  torch.empty(shapes[1], dtype=torch.uint8, device=w.device))
    if rows == 0 or cols == 0:
        return q
    w2, ldw, _ = _strided_rows(w, cols)
    d = q.descriptor()
    _launch(w.device, _lib.lib().qlora_fp8_quantize, _ptr(w2), ldw, code, ctypes.byref(d))
    return q


@functools.lru_cache(maxsize=4096)
def _fp8_bytes(rows, cols, m, code):
    d = QloraFp8(rows, cols, 0, None, None)
    return int(_lib.lib().qlora_fp8_workspace_bytes(ctypes.byref(d), m, code))


def fp8_workspace_bytes(w: Fp8Weight, m: int, dtype) -> int:
    """Workspace bytes of linear_fp8 on m tokens of ``dtype``."""
    return _fp8_bytes(w.rows, w.cols, m, dtype_code(dtype))


def linear_fp8(w: Fp8Weight, x, bias=None, out=None, workspace=None):
    """y = x . W^T (+ bias) in 8-bit floats: each block of 128 columns of a row of x gets a scale
    of its own and is brought to 8 bits within the call, the products are summed in fp32, y has x's
    dtype.  Leading dims of x are flattened to tokens; rows of x may be strided.  ``out`` may
    supply a preallocated output, which must not overlap x."""
    torch = _torch()
    dt, device = x.dtype, x.device
    code = dtype_code(dt)
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if w.codes.device != device:
        raise ValueError("w is on %s, x on %s" % (w.codes.device, device))
    x2, ldx, lead = _strided_rows(x, w.cols)
    m = x2.shape[0]
    if out is None:
        y = torch.empty(m, w.rows, dtype=dt, device=device)
    else:
        _check_tensor("out", out, device, dt, m * w.rows)
        y = out
    if bias is not None:
        _check_tensor("bias", bias, device, dt, w.rows)
    d = ctypes.byref(w.descriptor())
    ws = _workspace_on(device, _fp8_bytes(w.rows, w.cols, m, code), workspace)
    _launch(device, _lib.lib().qlora_fp8_linear, d, x2.data_ptr(), m, ldx, _ptr(bias), code, y.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size())
    if lead is None and y.dim() == 2:
        return y if y.shape[1] == w.rows else y.view(m, w.rows)
    return y.view(*((m,) if lead is None else lead), w.rows)


def distill_loss_grad(logits, top_values, top_index, temperature: float = 1.0, weight=None, need_grad: bool = True,
                      dlogits=None, row_kl=None, workspace=None):
    """loss = sum_i w_i T^2 KL(softmax(top_values_i / T) || softmax(logits_i / T)) (a 1-element
    fp32 GPU tensor) and its gradient with respect to the logits in their dtype (None without
    ``need_grad``).  logits [..., vocab] (rows may be strided); the teacher's logits top_values
    [..., k] (fp32, bf16 or f16) at the vocabulary entries top_index [..., k] (int32 or int64;
    -1, or a value of -inf, marks an absent slot).  ``weight`` [...] fp32 (default 1 / rows;
    0 leaves a row out); ``dlogits`` may be preallocated, ``logits`` itself included;
    ``row_kl`` (fp32, one per row) receives the rows' T^2 KL."""
    torch = _torch()
    dt, device = logits.dtype, logits.device
    code = dtype_code(dt)
    vocab = logits.shape[-1]
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    z, ldz, _ = _strided_rows(logits, vocab)
    n = z.shape[0]
    k = top_values.shape[-1]
    if k < 1:
        raise ValueError("top_values needs at least one slot per row")
    if top_index.dtype not in (torch.int32, torch.int64):
        raise TypeError("top_index must be int32 or int64, got %s" % (top_index.dtype,))
    u, ix = top_values, top_index
    if u.dim() != 2 or ix.dim() != 2:
        u, ix = u.reshape(-1, k), ix.reshape(-1, ix.shape[-1])
    if u.shape != (n, k) or ix.shape != (n, k):
        raise ValueError("top_values and top_index must be [%d rows, k]" % n)
    if u.device != device or ix.device != device:
        raise ValueError("top_values and top_index must be on %s" % (device,))
    u, ix = u.contiguous(), ix.contiguous()
    td = dtype_code(u.dtype)
    if weight is not None:
        _check_tensor("weight", weight, device, torch.float32, n)
    if row_kl is not None:
        _check_tensor("row_kl", row_kl, device, torch.float32, n)
    g, ldd = None, vocab
    if dlogits is not None:
        if not need_grad:
            raise ValueError("dlogits given without need_grad")
        if not dlogits.is_cuda or dlogits.dtype != dt or dlogits.shape != logits.shape or dlogits.device != device:
            raise ValueError("dlogits must be a GPU tensor like logits")
        d2, ldd, _ = _strided_rows(dlogits, vocab)
        if n and d2.data_ptr() != dlogits.data_ptr():
            raise ValueError("dlogits must have rows of contiguous elements, evenly spaced")
        g = dlogits
    elif need_grad:
        g = torch.empty_like(logits, memory_format=torch.contiguous_format)
    loss = torch.empty(1, dtype=torch.float32, device=device)
    lib = _lib.lib()
    ws = _workspace_on(device, lib.qlora_distill_workspace_bytes(n, vocab, k, code), workspace)
    _launch(device, lib.qlora_distill_loss_grad, z.data_ptr(), n, vocab, ldz, code, u.data_ptr(), td, ix.data_ptr(),
            64 if ix.dtype == torch.int64 else 32, k, float(temperature), _ptr(weight), loss.data_ptr(),
            _ptr(row_kl), _ptr(g), ldd, ws.data_ptr(), ws.numel() * ws.element_size())
    return loss, g


def _adamw(lr, beta1, beta2, eps, weight_decay):
    return _lib.QloraAdamW(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay))


def adamw_step(param, grad, m, v, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999,
               eps: float = 1e-8, weight_decay: float = 0.0, param_cd=None):
    """One in-place AdamW update of fp32 ``param`` (moments ``m``, ``v``; 1-based ``step``);
    ``param_cd`` (bf16 / f16 / fp32, optional) receives the rounded copy."""
    torch = _torch()
    for name, t in (("param", param), ("grad", grad), ("m", m), ("v", v)):
        _need_cuda(name, t, torch.float32)
        if t.numel() != param.numel():
            raise ValueError("%s has %d elements, param %d" % (name, t.numel(), param.numel()))
    cd = _lib.QLORA_F32
    if param_cd is not None:
        _need_cuda("param_cd", param_cd)
        cd = dtype_code(param_cd.dtype)
        if param_cd.numel() != param.numel():
            raise ValueError("param_cd has the wrong size")
    o = _adamw(lr, beta1, beta2, eps, weight_decay)
    _lib.check(_lib.lib().qlora_adamw_step(_ptr(param), _ptr(grad), _ptr(m), _ptr(v), param.numel(),
                                           ctypes.byref(o), int(step), _ptr(param_cd), cd,
                                           _stream_ptr(param.device)))


@dataclass
class StackLayer:
    """One layer of a trainable stack: frozen NF4 base, fp32 master adapters, their
    compute-dtype copies, AdamW moments and the gradient buffers the step writes."""
    q: NF4Weight
    lora_a: "object"
    lora_b: "object"
    a32: "object"
    b32: "object"
    m_a: "object"
    v_a: "object"
    m_b: "object"
    v_b: "object"
    grad_a: "object"
    grad_b: "object"

    @staticmethod
    def create(q: NF4Weight, a32, b32, dtype) -> "StackLayer":
        torch = _torch()
        a32 = a32.to(device=q.device, dtype=torch.float32).contiguous().clone()
        b32 = b32.to(device=q.device, dtype=torch.float32).contiguous().clone()
        z = torch.zeros_like
        return StackLayer(q, a32.to(dtype), b32.to(dtype), a32, b32, z(a32), z(a32), z(b32), z(b32), z(a32),
                          z(b32))

    @property
    def r(self) -> int:
        return self.a32.shape[0]

    def _struct(self, desc):
        return _lib.QloraStackLayer(ctypes.pointer(desc), *[_ptr(t) for t in (
            self.lora_a, self.lora_b, self.a32, self.b32, self.m_a, self.v_a, self.m_b, self.v_b,
            self.grad_a, self.grad_b)])


def _stack_structs(layers):
    descs = [L.q.descriptor() for L in layers]
    arr = (_lib.QloraStackLayer * len(layers))(*[L._struct(d) for L, d in zip(layers, descs)])
    return arr, descs


def stack_workspace_bytes(layers, m: int, dtype, rslora: bool = False, path: str = "auto") -> int:
    arr, _descs = _stack_structs(layers)
    return int(_lib.lib().qlora_stack_workspace_bytes(arr, len(layers), m, layers[0].r, dtype_code(dtype),
                                                      _flags(rslora, path)))


def stack_train_step(layers, x, target, alpha: float, step: int, lr: float, beta1: float = 0.9,
                     beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0, rslora: bool = False,
                     path: str = "auto", workspace=None, loss=None):
    """Forward through the stack, MSE loss against ``target``, backward, AdamW on every
    adapter (in place).  Returns the loss as a 1-element fp32 GPU tensor."""
    torch = _torch()
    dt = x.dtype
    x2, _ = _flatten(x, layers[0].q.cols)
    t2, _ = _flatten(target, layers[-1].q.rows)
    x2, t2 = x2.contiguous(), t2.contiguous()
    _need_cuda("x", x2, dt)
    _need_cuda("target", t2, dt)
    m = x2.shape[0]
    if t2.shape[0] != m:
        raise ValueError("target has %d rows, x %d" % (t2.shape[0], m))
    for L in layers:
        _need_cuda("lora_a", L.lora_a, dt)
        _need_cuda("lora_b", L.lora_b, dt)
    arr, _descs = _stack_structs(layers)
    flags = _flags(rslora, path)
    nbytes = int(_lib.lib().qlora_stack_workspace_bytes(arr, len(layers), m, layers[0].r, dtype_code(dt), flags))
    ws = _workspace(nbytes, x.device, workspace)
    loss = loss if loss is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    o = _adamw(lr, beta1, beta2, eps, weight_decay)
    _lib.check(_lib.lib().qlora_stack_train_step(arr, len(layers), _ptr(x2), m, _ptr(t2), layers[0].r, float(alpha),
                                                 flags, dtype_code(dt), ctypes.byref(o), int(step), _ptr(loss),
                                                 _ptr(ws), ws.numel() * ws.element_size(), _stream_ptr(x.device)))
    return loss


def levels():
    """The 16 fp32 NF4 levels the kernels use (host copy)."""
    out = (ctypes.c_float * 16)()
    _lib.check(_lib.lib().qlora_nf4_levels(out))
    return [float(v) for v in out]


def profile_enable(on: bool = True) -> None:
    """Start (resetting the totals) or stop per-kernel event timing in the library."""
    _lib.check(_lib.lib().qlora_profile_enable(1 if on else 0))


def profile_read():
    """{kernel kind: (summed milliseconds, launches)} recorded since profile_enable."""
    out = {}
    for kind, name in enumerate(_lib.KERNEL_KINDS):
        ms = ctypes.c_double()
        n = ctypes.c_int64()
        _lib.check(_lib.lib().qlora_profile_read(kind, ctypes.byref(ms), ctypes.byref(n)))
        out[name] = (ms.value, n.value)
    return out
