"""ctypes binding of libsp24.so (argument marshalling only).

Each function takes and returns torch tensors on the current HIP device; the
C library does all of the computing, on the caller's current torch stream.
Output tensors are allocated with torch when not supplied.  Errors from the
library raise :class:`Sp24Error`.  There is no fallback: without the built
library every call raises.

Shapes and layouts follow ``include/sp24.h``: W is fp16 [R, C]; idx uint8
[R/4, C/4]; the row form is (vals_row fp16 [R, C/2], meta_row int16 [R, C/16])
and the column form (vals_col fp16 [C, R/2], meta_col int16 [C, R/16]).  torch
has no uint16, so meta words travel as int16 tensors with the same bits.  The
forms' tensors carry those logical shapes, but their elements are in the
header's blocked order (64-row bands of contiguous column blocks), so a row
of such a tensor is not a row of the form.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsp24.so")

SP24_OK = 0
STATUS_NAMES = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_ALIGN", 4: "ERR_LAUNCH",
                5: "ERR_UNSUPPORTED", 6: "ERR_TOO_LARGE", 7: "ERR_WORKSPACE"}
EXPORTS = ("sp24_mask_search", "sp24_compress", "sp24_search_compress", "sp24_search_compress_batch",
           "sp24_flip_count", "sp24_weight_grad", "sp24_geglu_fwd", "sp24_geglu_bwd", "sp24_mvue",
           "sp24_spmm_fwd", "sp24_spmm_fwd_geglu", "sp24_spmm_bwd_input", "sp24_spmm_group",
           "sp24_spmm_group_noalloc", "sp24_embed_fwd", "sp24_embed_bwd", "sp24_embed_bwd_workspace",
           "sp24_orthogonalize", "sp24_orthogonalize_workspace", "sp24_muon_step", "sp24_muon_workspace",
           "sp24_spmm_fwd_act", "sp24_spmm_fwd_act_workspace", "sp24_spmm_bwd_input_act", "sp24_spmm_bwd_input_act_workspace",
           "sp24_bias_grad", "sp24_bias_grad_workspace", "sp24_grad_norm", "sp24_grad_norm_workspace",
           "sp24_adamw_step", "sp24_state8_values",
           "sp24_status_str",
           "sp24_pattern_table", "sp24_abi_version")
MAX_BATCH = 8
MAX_GROUP = 8
GROUP_WORKSPACE_BYTES = 64
MAX_NS_STEPS = 32
F16, F32, I32, I64, BF16, STATE8 = 0, 1, 2, 3, 4, 5
# SP24_ACT_*, by name
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}
FP16_OPERANDS = 16
# the usual quintic of the Newton-Schulz iteration: five steps bring singular
# values to about [0.7, 1.2]
NS_COEFFS = (3.4445, -4.7750, 2.0315)


class ScJob(ctypes.Structure):
    """Mirror of sp24_sc_job (include/sp24.h)."""
    _fields_ = [("W", ctypes.c_void_p), ("R", ctypes.c_int64), ("C", ctypes.c_int64), ("idx", ctypes.c_void_p),
                ("vals_row", ctypes.c_void_p), ("meta_row", ctypes.c_void_p),
                ("vals_col", ctypes.c_void_p), ("meta_col", ctypes.c_void_p),
                ("idx_prev", ctypes.c_void_p), ("flips", ctypes.c_void_p)]


class Gemm(ctypes.Structure):
    """Mirror of sp24_gemm (include/sp24.h)."""
    _fields_ = [("A", ctypes.c_void_p), ("vals", ctypes.c_void_p), ("meta", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("T", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class OrthoJob(ctypes.Structure):
    """Mirror of sp24_ortho_job (include/sp24.h)."""
    _fields_ = [("G", ctypes.c_void_p), ("out", ctypes.c_void_p), ("R", ctypes.c_int64), ("C", ctypes.c_int64)]


class MuonJob(ctypes.Structure):
    """Mirror of sp24_muon_job (include/sp24.h)."""
    _fields_ = [("G", ctypes.c_void_p), ("M", ctypes.c_void_p), ("P", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("R", ctypes.c_int64), ("C", ctypes.c_int64), ("lr", ctypes.c_float), ("decay", ctypes.c_float)]


class AdamwJob(ctypes.Structure):
    """Mirror of sp24_adamw_job (include/sp24.h)."""
    _fields_ = [("G", ctypes.c_void_p), ("P", ctypes.c_void_p), ("M", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("M_exps", ctypes.c_void_p), ("V_exps", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("lr", ctypes.c_float), ("decay", ctypes.c_float)]


class Sp24Error(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} ({text})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libsp24.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m structured_sparse_transformer_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        sig = {
            "sp24_mask_search": [p, i64, i64, p, p],
            "sp24_compress": [p, p, i64, i64, p, p, p, p, p],
            "sp24_search_compress": [p, i64, i64, p, p, p, p, p, p],
            "sp24_search_compress_batch": [p, i32, p],
            "sp24_flip_count": [p, p, i64, p, p],
            "sp24_weight_grad": [p, p, p, p, ctypes.c_float, i64, i64, i64, p, p],
            "sp24_geglu_fwd": [p, i64, i64, i64, p, p],
            "sp24_geglu_bwd": [p, p, i64, i64, i64, p, p],
            "sp24_mvue": [p, p, i64, i64, p, p, p],
            "sp24_spmm_fwd": [p, p, p, i64, i64, i64, p, p],
            "sp24_spmm_fwd_geglu": [p, p, p, i64, i64, i64, p, p, p],
            "sp24_spmm_bwd_input": [p, p, p, i64, i64, i64, p, p],
            "sp24_spmm_group": [p, i32, p, p],
            "sp24_spmm_group_noalloc": [p, i32, p],
            "sp24_embed_fwd": [p, i32, i64, p, i32, i64, i64, ctypes.c_float, p, p],
            "sp24_embed_bwd": [p, i32, i64, p, i64, i64, ctypes.c_float, i32, p, p, i64, p],
            "sp24_embed_bwd_workspace": [i64, i64, i64],
            "sp24_orthogonalize": [p, i32, i32, i32, p, i32, ctypes.c_float, p, i64, p],
            "sp24_orthogonalize_workspace": [p, i32],
            "sp24_muon_step": [p, i32, ctypes.c_float, i32, i32, p, i32, ctypes.c_float, p, i64, p],
            "sp24_muon_workspace": [p, i32],
            "sp24_spmm_fwd_act": [p, p, p, i64, i64, i64, p, i32, p, p, p, p, i64, p],
            "sp24_spmm_fwd_act_workspace": [i64, i64, i64],
            "sp24_spmm_bwd_input_act": [p, p, p, i64, i64, i64, i32, p, p, p, p, i64, p],
            "sp24_spmm_bwd_input_act_workspace": [i64, i64, i64],
            "sp24_bias_grad": [p, i64, i64, p, p, i64, p],
            "sp24_bias_grad_workspace": [i64, i64],
            "sp24_grad_norm": [p, p, i64, i32, ctypes.c_float, ctypes.c_float, p, p, i64, p],
            "sp24_grad_norm_workspace": [p, i64],
            "sp24_adamw_step": [p, i64, i32, i32, ctypes.c_double, ctypes.c_double, ctypes.c_double, i64, p,
                                ctypes.c_uint32, p],
            "sp24_state8_values": [p, p, i64, i32, i32, p, p],
            "sp24_status_str": [i32],
            "sp24_pattern_table": [p],
            "sp24_abi_version": [],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = (ctypes.c_char_p if name == "sp24_status_str" else
                         i64 if name.endswith("_workspace") else i32)
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != SP24_OK:
        raise Sp24Error(fn, status, lib().sp24_status_str(status).decode())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    # the library launches on the current device (and its current stream)
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"tensor is on {t.device} but the current device is cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr()) if t.numel() else None


def _stream(stream):
    if stream is None:   # its handle alone: a Stream object would cost more than a launch
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    s = stream
    if s.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {s.device} but the current device is cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(s.cuda_stream)


def _out(t, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"output must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def _need(t, shape, dtype, name):
    """An input tensor the library reads through a plain pointer: its shape and
    dtype must be exactly what the sizes passed alongside it imply, or the
    kernels would read past its end."""
    if t is None or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        got = "None" if t is None else f"{t.dtype} {tuple(t.shape)}"
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {got}")
    return t


def _row_form(vals, meta, R, C, name):
    """The 2:4 form of an [R, C] matrix: vals fp16 [R, C/2], meta int16 [R, C/16]."""
    if R % 16 or C % 16:
        raise ValueError(f"{name}: both dimensions must be multiples of 16, got {R} x {C}")
    _need(vals, (R, C // 2), torch.float16, f"{name} values")
    _need(meta, (R, C // 16), torch.int16, f"{name} metadata")


def _w(W):
    if W.dtype != torch.float16 or W.dim() != 2:
        raise ValueError("W must be a 2-D float16 tensor")
    return W.shape


def sp24_mask_search(W, idx=None, stream=None):
    """idx[R/4, C/4] (uint8) of the transposable pattern kept by each 4x4 block."""
    R, C = _w(W)
    idx = _out(idx, (R // 4, C // 4), torch.uint8, W.device)
    _check("sp24_mask_search", lib().sp24_mask_search(_ptr(W), R, C, _ptr(idx), _stream(stream)))
    return idx


def _forms(R, C, device, row, col, out):
    out = dict(out or {})
    if row:
        out["vals_row"] = _out(out.get("vals_row"), (R, C // 2), torch.float16, device)
        out["meta_row"] = _out(out.get("meta_row"), (R, C // 16), torch.int16, device)
    if col:
        out["vals_col"] = _out(out.get("vals_col"), (C, R // 2), torch.float16, device)
        out["meta_col"] = _out(out.get("meta_col"), (C, R // 16), torch.int16, device)
    return out


def sp24_compress(W, idx, row=True, col=True, out=None, stream=None):
    """Row and/or column 2:4 forms of W pruned by the masks ``idx``."""
    R, C = _w(W)
    _need(idx, (R // 4, C // 4), torch.uint8, "idx")
    o = _forms(R, C, W.device, row, col, out)
    _check("sp24_compress", lib().sp24_compress(
        _ptr(W), _ptr(idx), R, C, _ptr(o.get("vals_row")), _ptr(o.get("meta_row")),
        _ptr(o.get("vals_col")), _ptr(o.get("meta_col")), _stream(stream)))
    return o


def sp24_search_compress(W, want_idx=True, row=True, col=True, out=None, stream=None):
    """Mask search and compression in one pass over W."""
    R, C = _w(W)
    o = _forms(R, C, W.device, row, col, out)
    if want_idx:
        o["idx"] = _out(o.get("idx"), (R // 4, C // 4), torch.uint8, W.device)
    _check("sp24_search_compress", lib().sp24_search_compress(
        _ptr(W), R, C, _ptr(o.get("idx")), _ptr(o.get("vals_row")), _ptr(o.get("meta_row")),
        _ptr(o.get("vals_col")), _ptr(o.get("meta_col")), _stream(stream)))
    return o


def _flip_counter(f):
    """A uint64 flip counter travels as an int64 tensor view of one element."""
    if f is None:
        return None
    if f.dtype != torch.int64 or f.numel() != 1:
        raise ValueError("a flip counter is a one-element int64 tensor (or a view of one)")
    return _ptr(f).value


def sp24_search_compress_batch(Ws, outs=None, want_idx=True, row=True, col=True, prev=None, flips=None,
                               stream=None):
    """sp24_search_compress for several weights in one launch; returns one dict per weight.

    ``prev[k]`` (uint8 [R/4, C/4]) and ``flips[k]`` (a one-element int64 tensor)
    make weight k count its flipped mask entries against ``prev[k]``: the
    count is ADDED to ``flips[k]``.  ``prev[k]`` may be the weight's own
    ``outs[k]["idx"]``, which is then updated in place.
    """
    if not 1 <= len(Ws) <= MAX_BATCH:
        raise ValueError(f"between 1 and {MAX_BATCH} weights per batch")
    outs = list(outs) if outs is not None else [None] * len(Ws)
    prev = list(prev) if prev is not None else [None] * len(Ws)
    flips = list(flips) if flips is not None else [None] * len(Ws)
    if len(prev) != len(Ws) or len(flips) != len(Ws):
        raise ValueError("prev and flips need one entry per weight")
    res, jobs = [], (ScJob * len(Ws))()
    for k, W in enumerate(Ws):
        R, C = _w(W)
        o = _forms(R, C, W.device, row, col, outs[k])
        if want_idx:
            o["idx"] = _out(o.get("idx"), (R // 4, C // 4), torch.uint8, W.device)
        ptr = lambda t: _ptr(t).value if t is not None and t.numel() else None  # noqa: E731
        if prev[k] is not None:
            _need(prev[k], (R // 4, C // 4), torch.uint8, "prev")
        jobs[k] = ScJob(ptr(W), R, C, ptr(o.get("idx")), ptr(o.get("vals_row")), ptr(o.get("meta_row")),
                        ptr(o.get("vals_col")), ptr(o.get("meta_col")), ptr(prev[k]), _flip_counter(flips[k]))
        res.append(o)
    _check("sp24_search_compress_batch",
           lib().sp24_search_compress_batch(ctypes.cast(jobs, ctypes.c_void_p), len(Ws), _stream(stream)))
    return res


def sp24_flip_count(idx_prev, idx_new, flips=None, stream=None):
    """Adds to ``flips`` (a one-element int64 tensor, zeroed when not given)
    the number of mask entries that differ between the two index arrays."""
    if idx_prev.dtype != torch.uint8 or idx_new.dtype != torch.uint8 or idx_prev.shape != idx_new.shape:
        raise ValueError("idx_prev and idx_new must be uint8 tensors of one shape")
    if flips is None:
        flips = torch.zeros(1, dtype=torch.int64, device=idx_new.device)
    _check("sp24_flip_count", lib().sp24_flip_count(_ptr(idx_prev), _ptr(idx_new), idx_new.numel(),
                                                    _flip_counter(flips), _stream(stream)))
    return flips


def sp24_weight_grad(dY, X, W=None, idx=None, decay=0.0, dW=None, stream=None):
    """dW[R, C] (float32) = dY^T X + decay * (1 - M) * W, M the masks ``idx``."""
    T, R = dY.shape
    C = X.shape[1]
    if dY.dtype != torch.float16 or X.dtype != torch.float16 or X.dim() != 2 or X.shape[0] != T:
        raise ValueError("dY and X must be float16 [T, R] and [T, C]")
    if W is not None:
        _need(W, (R, C), torch.float16, "W")
    if idx is not None:
        _need(idx, (R // 4, C // 4), torch.uint8, "idx")
    dW = _out(dW, (R, C), torch.float32, dY.device)
    _check("sp24_weight_grad", lib().sp24_weight_grad(_ptr(dY), _ptr(X), _ptr(W), _ptr(idx), float(decay), T, R, C,
                                                      _ptr(dW), _stream(stream)))
    return dW


def _geglu_shape(U, group):
    if U.dtype != torch.float16 or U.dim() != 2 or U.shape[1] % 2:
        raise ValueError("U must be float16 [T, 2h]")
    T, h = U.shape[0], U.shape[1] // 2
    group = h if group is None else group
    return T, h, group


def sp24_geglu_fwd(U, group=None, out=None, stream=None):
    """out [T, h] = value * GELU(gate); U's columns in blocks of `group`
    values then `group` gates (default: the two halves)."""
    T, h, group = _geglu_shape(U, group)
    out = _out(out, (T, h), torch.float16, U.device)
    _check("sp24_geglu_fwd", lib().sp24_geglu_fwd(_ptr(U), T, h, group, _ptr(out), _stream(stream)))
    return out


def sp24_geglu_bwd(U, dout, group=None, dU=None, stream=None):
    """dU [T, 2h] in U's layout from dout [T, h]."""
    T, h, group = _geglu_shape(U, group)
    if dout.dtype != torch.float16 or tuple(dout.shape) != (T, h):
        raise ValueError("dout must be float16 [T, h]")
    dU = _out(dU, (T, 2 * h), torch.float16, U.device)
    _check("sp24_geglu_bwd", lib().sp24_geglu_bwd(_ptr(U), _ptr(dout), T, h, group, _ptr(dU), _stream(stream)))
    return dU


def sp24_mvue(M, U, out=None, stream=None):
    """MVUE 2:4 estimate of M (fp16 [rows, cols]) with uniforms U (fp32
    [rows, cols/4]); returns {"vals": fp16 [rows, cols/2], "meta": int16
    [rows, cols/16]}."""
    if M.dtype != torch.float16 or M.dim() != 2:
        raise ValueError("M must be a 2-D float16 tensor")
    rows, cols = M.shape
    if U.dtype != torch.float32 or tuple(U.shape) != (rows, cols // 4):
        raise ValueError("U must be float32 [rows, cols/4]")
    out = dict(out or {})
    out["vals"] = _out(out.get("vals"), (rows, cols // 2), torch.float16, M.device)
    out["meta"] = _out(out.get("meta"), (rows, cols // 16), torch.int16, M.device)
    _check("sp24_mvue", lib().sp24_mvue(_ptr(M), _ptr(U), rows, cols, _ptr(out["vals"]), _ptr(out["meta"]),
                                        _stream(stream)))
    return out


def sp24_spmm_fwd(X, vals_row, meta_row, R, C, Y=None, stream=None):
    """Y[T, R] = X[T, C] * Ws^T."""
    T = X.shape[0]
    if X.dtype != torch.float16 or tuple(X.shape) != (T, C):
        raise ValueError("X must be float16 [T, C]")
    _row_form(vals_row, meta_row, R, C, "the row form")
    Y = _out(Y, (T, R), torch.float16, X.device)
    _check("sp24_spmm_fwd", lib().sp24_spmm_fwd(_ptr(X), _ptr(vals_row), _ptr(meta_row), T, R, C,
                                                _ptr(Y), _stream(stream)))
    return Y


def sp24_spmm_fwd_geglu(X, vals_row, meta_row, R, C, out=None, U=False, stream=None):
    """out[T, R/2] = value * GELU(gate) of U = X * Ws^T, W's rows in blocks of
    16 values then their 16 gates.  U=True also returns the products [T, R]
    (a tensor may be passed instead); returns (out, U or None)."""
    T = X.shape[0]
    if X.dtype != torch.float16 or tuple(X.shape) != (T, C):
        raise ValueError("X must be float16 [T, C]")
    _row_form(vals_row, meta_row, R, C, "the row form")
    out = _out(out, (T, R // 2), torch.float16, X.device)
    if U is True:
        U = torch.empty(T, R, dtype=torch.float16, device=X.device)
    elif U is False or U is None:
        U = None
    else:
        U = _out(U, (T, R), torch.float16, X.device)
    _check("sp24_spmm_fwd_geglu", lib().sp24_spmm_fwd_geglu(_ptr(X), _ptr(vals_row), _ptr(meta_row), T, R, C,
                                                            _ptr(U), _ptr(out), _stream(stream)))
    return out, U


def sp24_spmm_bwd_input(dY, vals_col, meta_col, R, C, dX=None, stream=None):
    """dX[T, C] = dY[T, R] * Ws."""
    T = dY.shape[0]
    if dY.dtype != torch.float16 or tuple(dY.shape) != (T, R):
        raise ValueError("dY must be float16 [T, R]")
    _row_form(vals_col, meta_col, C, R, "the column form")
    dX = _out(dX, (T, C), torch.float16, dY.device)
    _check("sp24_spmm_bwd_input", lib().sp24_spmm_bwd_input(_ptr(dY), _ptr(vals_col), _ptr(meta_col), T, R, C,
                                                            _ptr(dX), _stream(stream)))
    return dX


def sp24_pattern_table():
    """The 90 patterns as 16-bit masks (bit 4r+c for kept entry (r, c))."""
    buf = (ctypes.c_uint16 * 90)()
    _check("sp24_pattern_table", lib().sp24_pattern_table(ctypes.cast(buf, ctypes.c_void_p)))
    return list(buf)


_group_ws = {}


def group_workspace(device=None):
    """The binding's workspace for sp24_spmm_group on a device: zeroed once,
    and left zero by every call that completes.  Calls that overlap in time
    (on different streams) must pass workspaces of their own."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index)
    ws = _group_ws.get(dev.index)
    if ws is None:
        ws = torch.zeros(GROUP_WORKSPACE_BYTES // 4, dtype=torch.int32, device=dev)
        _group_ws[dev.index] = ws
    return ws


def _gemm_descs(gemms):
    if not 1 <= len(gemms) <= MAX_GROUP:
        raise ValueError(f"between 1 and {MAX_GROUP} products per group")
    descs, outs = (Gemm * len(gemms))(), []
    for k, (A, vals, meta, out) in enumerate(gemms):
        if A.dtype != torch.float16 or A.dim() != 2:
            raise ValueError("A must be a 2-D float16 tensor")
        T, K = A.shape
        if vals.dim() != 2:
            raise ValueError("vals must be 2-D")
        N = vals.shape[0]
        _row_form(vals, meta, N, K, f"product {k}")
        out = _out(out, (T, N), torch.float16, A.device)
        outs.append(out)
        ptr = lambda t: _ptr(t).value if t is not None and t.numel() else None  # noqa: E731
        descs[k] = Gemm(ptr(A), ptr(vals), ptr(meta), ptr(out), T, N, K)
    return descs, outs


def sp24_spmm_group_noalloc(gemms, stream=None):
    """sp24_spmm_group with the library's own per-GPU queue counters instead
    of a workspace (the C entry point allocates nothing).  Calls that overlap
    in time on one GPU race.  Output tensors given as None are allocated here
    by torch; pass them all to keep the whole call allocation-free."""
    descs, outs = _gemm_descs(gemms)
    _check("sp24_spmm_group_noalloc", lib().sp24_spmm_group_noalloc(ctypes.cast(descs, ctypes.c_void_p), len(gemms),
                                                                    _stream(stream)))
    return outs


def sp24_spmm_group(gemms, workspace=None, stream=None):
    """Several independent products out = A * S^T in one launch.

    ``gemms`` is a list of (A, vals, meta, out) with A fp16 [T, K], (vals,
    meta) the 2:4 row form of S [N, K] (fp16 [N, K/2], int16 [N, K/16]) and
    out fp16 [T, N] or None (allocated).  The forward product of a layer is
    (X, vals_row, meta_row, Y); its input gradient (dY, vals_col, meta_col,
    dX).  Returns the outputs."""
    descs, outs = _gemm_descs(gemms)
    ws = group_workspace() if workspace is None else workspace
    if ws.numel() * ws.element_size() < GROUP_WORKSPACE_BYTES:
        raise ValueError(f"the workspace needs {GROUP_WORKSPACE_BYTES} bytes")
    _check("sp24_spmm_group", lib().sp24_spmm_group(ctypes.cast(descs, ctypes.c_void_p), len(gemms), _ptr(ws),
                                                    _stream(stream)))
    return outs


def _id_type(ids):
    types = {torch.int32: I32, torch.int64: I64}
    if ids.dtype not in types:
        raise ValueError("ids must be int32 or int64")
    return types[ids.dtype]


_HERE_AND_NOW = contextlib.nullcontext()


def _using(stream):
    """What is allocated within belongs to the stream that the call runs on."""
    return _HERE_AND_NOW if stream is None else torch.cuda.stream(stream)


def _workspace(t, need, device):
    """The caller's workspace, or one of `need` bytes."""
    if need < 0:
        raise ValueError("the sizes are beyond what the call takes")
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if t.numel() * t.element_size() < need:
        raise ValueError(f"the workspace needs {need} bytes")
    return t


def _laid_out(ids, stream):
    """ids as the library takes them.  A part of a token stream may start at any
    id, and a batch's inputs and targets are views of one tensor: those are copied."""
    if ids.is_contiguous() and ids.data_ptr() % 16 == 0:
        return ids
    with _using(stream):
        return ids.clone(memory_format=torch.contiguous_format)


def sp24_embed_fwd(ids, table, scale=1.0, out=None, stream=None):
    """out [*ids.shape, d] (float16) = scale * table[ids]; rows of ids outside
    [0, V) are zeros.  ids int32 or int64, of any strides; table float16 or
    float32 [V, d]."""
    types = {torch.float16: F16, torch.float32: F32}
    if table.dtype not in types or table.dim() != 2:
        raise ValueError("the table must be a 2-D float16 or float32 tensor")
    kind = _id_type(ids)
    V, d = table.shape
    ids = _laid_out(ids, stream)
    with _using(stream):
        out = _out(out, (*ids.shape, d), torch.float16, table.device)
    _check("sp24_embed_fwd", lib().sp24_embed_fwd(_ptr(ids), kind, ids.numel(), _ptr(table), types[table.dtype], V, d,
                                                  float(scale), _ptr(out), _stream(stream)))
    return out


def sp24_embed_bwd_workspace(T, V, d):
    """Bytes of sp24_embed_bwd's workspace."""
    return lib().sp24_embed_bwd_workspace(T, V, d)


def sp24_embed_bwd(ids, dout, V, scale=1.0, dtable=None, accumulate=False, workspace=None, stream=None):
    """dtable [V, d] (float32): scale times the sums of dout's rows by id, in
    token order.  ``accumulate`` adds them to the ``dtable`` given."""
    kind = _id_type(ids)
    if dout.dtype != torch.float16 or dout.dim() != ids.dim() + 1 or dout.shape[:-1] != ids.shape:
        raise ValueError("dout must be float16 [*ids.shape, d]")
    if accumulate and dtable is None:
        raise ValueError("accumulate needs the dtable to add to")
    if V < 0:
        raise ValueError("V must not be negative")
    T, d = ids.numel(), dout.shape[-1]
    ids = _laid_out(ids, stream)
    with _using(stream):
        dtable = _out(dtable, (V, d), torch.float32, dout.device)
        workspace = _workspace(workspace, sp24_embed_bwd_workspace(T, V, d), dout.device)
    _check("sp24_embed_bwd", lib().sp24_embed_bwd(
        _ptr(ids), kind, T, _ptr(dout), V, d, float(scale), int(bool(accumulate)), _ptr(dtable), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dtable


def _coeffs(coeffs, steps):
    """The (a, b, c) of every step: one triple for all of them, or one each."""
    if not 1 <= steps <= MAX_NS_STEPS:
        raise ValueError(f"between 1 and {MAX_NS_STEPS} steps")
    rows = list(NS_COEFFS if coeffs is None else coeffs)
    try:
        rows = [[float(v) for v in r] for r in rows]
    except TypeError:   # numbers, not triples
        rows = [[float(v) for v in rows]] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coeffs must be (a, b, c), or one such triple per step")
    return (ctypes.c_float * (3 * steps))(*[v for r in rows for v in r])


def sp24_orthogonalize_batch(Gs, steps=5, coeffs=None, eps=1e-7, dtype=torch.float16, outs=None, workspace=None,
                             stream=None, precise=True):
    """The orthogonalised updates of up to 8 weights (all float16 or all
    float32, [R, C] each) by `steps` Newton-Schulz steps, in one sequence of
    launches.  The results are of ``dtype``, float16 or float32, computed to
    float32's accuracy and rounded once; ``precise=False`` takes products of
    fp16 operands, a third of the matrix work."""
    if not 1 <= len(Gs) <= MAX_BATCH:
        raise ValueError(f"between 1 and {MAX_BATCH} updates per batch")
    types = {torch.float16: F16, torch.float32: F32}
    if dtype not in types or any(G.dtype not in types or G.dtype != Gs[0].dtype or G.dim() != 2 for G in Gs):
        raise ValueError("updates must be 2-D float16 or float32 tensors of one type, dtype one of the two")
    coef = _coeffs(coeffs, steps)
    if outs is not None and len(outs) != len(Gs):
        raise ValueError("outs needs one entry per update")
    res, jobs = [], (OrthoJob * len(Gs))()
    for k, G in enumerate(Gs):
        with _using(stream):
            out = _out(outs[k] if outs is not None else None, G.shape, dtype, G.device)
        ptr = lambda t: _ptr(t).value if t.numel() else None  # noqa: E731
        jobs[k] = OrthoJob(ptr(G), ptr(out), G.shape[0], G.shape[1])
        res.append(out)
    arr = ctypes.cast(jobs, ctypes.c_void_p)
    with _using(stream):
        workspace = _workspace(workspace, lib().sp24_orthogonalize_workspace(arr, len(Gs)), Gs[0].device)
    _check("sp24_orthogonalize", lib().sp24_orthogonalize(
        arr, len(Gs), types[Gs[0].dtype], types[dtype] | (0 if precise else FP16_OPERANDS),
        ctypes.cast(coef, ctypes.c_void_p), steps, float(eps),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return res


def sp24_orthogonalize(G, steps=5, coeffs=None, eps=1e-7, dtype=torch.float16, out=None, workspace=None, stream=None,
                       precise=True):
    """sp24_orthogonalize_batch of one update."""
    return sp24_orthogonalize_batch([G], steps, coeffs, eps, dtype, None if out is None else [out], workspace, stream,
                                    precise)[0]


def sp24_muon_step(Gs, Ms, Ps, Ws, lrs, decays=None, momentum=0.95, nesterov=True, steps=5, coeffs=None, eps=1e-7,
                   precise=True, workspace=None, stream=None):
    """One optimiser step of up to 8 weights, in place: momentum Ms[k] and
    weights Ps[k] (float32 [R, C]) from the gradient Gs[k] (float32), and
    Ws[k] (float16, or None) = Ps[k].  lrs[k] multiplies the orthogonalised
    update, 1 - decays[k] the weight.  ``precise`` as sp24_orthogonalize_batch
    takes it."""
    n = len(Gs)
    if not 1 <= n <= MAX_BATCH:
        raise ValueError(f"between 1 and {MAX_BATCH} weights per step")
    decays = [0.0] * n if decays is None else decays
    if any(len(v) != n for v in (Ms, Ps, Ws, lrs, decays)):
        raise ValueError("Ms, Ps, Ws, lrs and decays need one entry per gradient")
    coef = _coeffs(coeffs, steps)
    jobs = (MuonJob * n)()
    ptr = lambda t: _ptr(t).value if t is not None and t.numel() else None  # noqa: E731
    for k, (G, M, P, W) in enumerate(zip(Gs, Ms, Ps, Ws)):
        if G.dtype != torch.float32 or G.dim() != 2:
            raise ValueError("gradients must be 2-D float32 tensors")
        _need(M, G.shape, torch.float32, "the momentum")
        _need(P, G.shape, torch.float32, "the weight")
        if W is not None:
            _need(W, G.shape, torch.float16, "the float16 weight")
        jobs[k] = MuonJob(ptr(G), ptr(M), ptr(P), ptr(W), G.shape[0], G.shape[1], float(lrs[k]), float(decays[k]))
    arr = ctypes.cast(jobs, ctypes.c_void_p)
    with _using(stream):
        workspace = _workspace(workspace, lib().sp24_muon_workspace(arr, n), Gs[0].device)
    _check("sp24_muon_step", lib().sp24_muon_step(
        arr, n, float(momentum), int(bool(nesterov)), int(bool(precise)), ctypes.cast(coef, ctypes.c_void_p), steps,
        float(eps), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def _act(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def _addresses(*tensors):
    """_ptr of a call's tensors, as plain numbers (0: NULL): a call of one token
    costs as much in here as on the GPU."""
    device, res = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else 0, []
    for t in tensors:
        if t is None:
            res.append(None)
            continue
        if t.get_device() != device:   # -1 for host memory
            _ptr(t)
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
        res.append(t.data_ptr() or None)
    return res


def _apart(outputs, inputs, in_place):
    """That the outputs which the caller passed share no memory with each other or
    with what other workgroups of the call may still read; the first of them may be
    the input `in_place` itself, where every entry is read and written by one lane."""
    span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())  # noqa: E731
    given = [t for t in outputs if isinstance(t, torch.Tensor)]
    for k, out in enumerate(given):
        a, b = span(out)
        own = in_place is not None and out is outputs[0] and a == in_place.data_ptr()
        for t in (*given[:k], *inputs, None if own else in_place):
            c, d = (0, 0) if t is None else span(t)
            if a < d and c < b:
                raise ValueError("an output shares memory with another tensor of the call")


def sp24_spmm_fwd_act(X, vals_row, meta_row, R, C, act="none", bias=None, residual=None, U=False, out=None,
                      workspace=None, stream=None):
    """Y [T, R] = act(U) + residual, U = X * Ws^T + bias (float32 [R]); each
    rounded once to float16.  U=True also returns U (a tensor may be passed
    instead); returns (Y, U or None).  ``out`` may be the residual, unless that is
    X; otherwise outputs share no memory with the call's other tensors."""
    kind, f16 = _act(act), torch.float16
    T = X.shape[0]
    if X.dtype != f16 or X.shape != (T, C):
        raise ValueError("X must be float16 [T, C]")
    _row_form(vals_row, meta_row, R, C, "the row form")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (R,)):
        _need(bias, (R,), torch.float32, "bias")
    if residual is not None and (residual.dtype != f16 or residual.shape != (T, R)):
        _need(residual, (T, R), f16, "residual")
    if out is not None or isinstance(U, torch.Tensor):
        _apart((out, U), (X, vals_row, meta_row, bias), residual)
    L = lib()
    with _using(stream):
        out = X.new_empty((T, R)) if out is None else _out(out, (T, R), f16, X.device)
        U = None if U is False or U is None else _out(None if U is True else U, (T, R), f16, X.device)
        need = L.sp24_spmm_fwd_act_workspace(T, R, C)
        workspace = _workspace(workspace, need, X.device) if need else None
    x, v, m, b, r, u, y, w = _addresses(X, vals_row, meta_row, bias, residual, U, out, workspace)
    _check("sp24_spmm_fwd_act", L.sp24_spmm_fwd_act(
        x, v, m, T, R, C, b, kind, r, u, y, w, 0 if w is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out, U


def sp24_spmm_bwd_input_act(dY, vals_col, meta_col, R, C, U, act="none", dbias=True, out=None, workspace=None,
                            stream=None):
    """dU [T, C] = (dY [T, R] * Ws) * act'(U) and dbias [C] (float32), dU's sums
    over tokens before they are rounded.  dbias=False leaves the sums out (a
    tensor may be passed instead).  ``out`` may be U, and U None without an
    activation; otherwise outputs share no memory with the call's other tensors.
    Returns (dU, dbias or None)."""
    kind, f16 = _act(act), torch.float16
    T = dY.shape[0]
    if dY.dtype != f16 or dY.shape != (T, R):
        raise ValueError("dY must be float16 [T, R]")
    _row_form(vals_col, meta_col, C, R, "the column form")
    if U is not None or kind:
        _need(U, (T, C), f16, "U")
    if out is not None or isinstance(dbias, torch.Tensor):
        _apart((out, dbias), (dY, vals_col, meta_col), U)
    L = lib()
    with _using(stream):
        out = _out(out, (T, C), f16, dY.device)
        dbias = None if dbias is False or dbias is None else _out(None if dbias is True else dbias, (C,), torch.float32,
                                                                  dY.device)
        need = L.sp24_spmm_bwd_input_act_workspace(T, R, C)
        workspace = _workspace(workspace, need, dY.device) if need else None
    y, v, m, u, o, b, w = _addresses(dY, vals_col, meta_col, U, out, dbias, workspace)
    _check("sp24_spmm_bwd_input_act", L.sp24_spmm_bwd_input_act(
        y, v, m, T, R, C, kind, u, o, b, w, 0 if w is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out, dbias


def sp24_bias_grad(dY, dbias=None, workspace=None, stream=None):
    """dbias [R] (float32): the sums of dY [T, R] (float16) over tokens."""
    if dY.dtype != torch.float16 or dY.dim() != 2:
        raise ValueError("dY must be float16 [T, R]")
    T, R = dY.shape
    L = lib()
    need = L.sp24_bias_grad_workspace(T, R)
    with _using(stream):
        dbias = _out(dbias, (R,), torch.float32, dY.device)
        workspace = _workspace(workspace, need, dY.device) if need else None
    y, b, w = _addresses(dY, dbias, workspace)
    _check("sp24_bias_grad", L.sp24_bias_grad(
        y, T, R, b, w, 0 if w is None else workspace.numel() * workspace.element_size(), _stream(stream)))
    return dbias


def step_control(device="cuda"):
    """What sp24_grad_norm writes and sp24_adamw_step reads (sp24_step_control),
    before the first step: int32 [8], zeros."""
    return torch.zeros(8, dtype=torch.int32, device=device)


def control_values(control):
    """Views of a control's fields: step (int64), norm, factor (float32), skip (int32)."""
    return {"step": control.view(torch.int64)[0], "norm": control.view(torch.float32)[2],
            "factor": control.view(torch.float32)[3], "skip": control[4]}


def _control(control):
    return _need(control, (8,), torch.int32, "the control")


def _gradients(grads):
    """Checks many gradients, each of _ptr's checks over all of them at once, and
    gives their type's number, addresses and sizes."""
    Tensor, types = torch.Tensor, {t.dtype for t in grads}
    if not types:
        return F32, [], []
    kind = {torch.float16: F16, torch.float32: F32}.get(types.pop())
    if kind is None or types:
        raise ValueError("gradients must be all float16 or all float32")
    if not all(map(Tensor.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous")
    devices = set(map(Tensor.get_device, grads))
    if -1 in devices or devices != {torch.cuda.current_device()}:   # -1: host memory
        raise ValueError("gradients must be on the current device")
    return kind, list(map(Tensor.data_ptr, grads)), list(map(Tensor.numel, grads))


def _int64s(values):
    """An array of 64-bit numbers that the library reads, and its address."""
    a = array.array("q", values)
    return a, a.buffer_info()[0] or None


def sp24_grad_norm(grads, scale=1.0, max_norm=float("inf"), control=None, workspace=None, stream=None):
    """The norm of all gradients together (all float16 or all float32, of any
    shapes) times ``scale``, and the factor that takes the scale off them and
    clips them to ``max_norm``, in a control (see step_control; one is made
    unless given), whose step grows by 1 unless some gradient is not finite."""
    kind, pointers, sizes = _gradients(grads)
    n, L = len(grads), lib()
    (pointers, at), (sizes, sizes_at) = _int64s(pointers), _int64s(sizes)
    with _using(stream):
        if control is None:
            control = step_control(torch.device("cuda", torch.cuda.current_device()))
        _control(control)
        workspace = _workspace(workspace, L.sp24_grad_norm_workspace(sizes_at, n), control.device)
    c, w = _addresses(control, workspace)
    _check("sp24_grad_norm", L.sp24_grad_norm(
        at, sizes_at, n, kind, float(scale), float(max_norm), c, w, workspace.numel() * workspace.element_size(), _stream(stream)))
    return control


class AdamwPlan:
    """The tensors of an AdamW step, checked once and laid out as the library
    takes them; sp24_adamw_plan makes one.  It holds the tensors."""

    def __init__(self, jobs, tensors, sizes, state8):
        self.jobs, self.tensors, self.sizes, self.state8 = jobs, tensors, sizes, state8
        self._shaped = [(k, P.shape) for k, P in enumerate(tensors[0]) if P.dim() > 1]
        self.address = ctypes.addressof(jobs) if sizes else None
        # the jobs' first fields, the gradients' addresses
        words = np.frombuffer(jobs, dtype=np.int64) if sizes else np.zeros(0, dtype=np.int64)
        self.gradients = words[::ctypes.sizeof(AdamwJob) // 8]

    def check(self, Gs, sizes):
        """That gradients of these sizes are the tensors'.  Not by sizes alone: the
        gradients of [h, d] and [d, h] weights could be taken for one another."""
        if sizes != self.sizes or any(Gs[k].shape != shape for k, shape in self._shaped):
            raise ValueError("one gradient per tensor, of its shape")


def sp24_adamw_plan(Ps, Ms, Vs, Ws=None, lrs=1e-3, decays=0.0, M_exps=None, V_exps=None):
    """The plan of sp24_adamw_step over tensors of any shapes: Ps float32; Ms and
    Vs float32, or uint8 with M_exps and V_exps (uint8, one for 64 entries: see
    state8); Ws float16 or None, or None altogether.  lrs and decays are one
    number for all tensors or one each; decays are the parts of Ps that a step
    takes off."""
    n = len(Ps)
    state8 = M_exps is not None
    if (V_exps is not None) != state8:
        raise ValueError("M_exps and V_exps are given together")
    Ws = [None] * n if Ws is None else Ws
    lrs, decays = ([float(v)] * n if isinstance(v, (int, float)) else [float(x) for x in v] for v in (lrs, decays))
    more = (M_exps, V_exps) if state8 else ()
    if any(len(v) != n for v in (Ms, Vs, Ws, lrs, decays, *more)):
        raise ValueError("every list needs one entry per tensor")
    sizes = [P.numel() for P in Ps]
    dtype = torch.uint8 if state8 else torch.float32
    for k, (P, M, V, W) in enumerate(zip(Ps, Ms, Vs, Ws)):
        _need(P, P.shape, torch.float32, "P")
        _need(M, P.shape, dtype, "M")
        _need(V, P.shape, dtype, "V")
        if W is not None:
            _need(W, P.shape, torch.float16, "W")
        if state8:
            _need(M_exps[k], (-(-sizes[k] // 64),), torch.uint8, "M_exps")
            _need(V_exps[k], (-(-sizes[k] // 64),), torch.uint8, "V_exps")
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for part in (Ps, Ms, Vs, Ws, *more)
                   for t in part if t is not None and t.numel())
    if any(end > start for (_, end), (start, _) in zip(spans, spans[1:])):
        raise ValueError("tensors of a plan share memory: a tensor takes one step, whichever layers use it")
    # here, since a step that the library refuses comes after the norm has counted it
    if any(t.data_ptr() % 16 for part in (Ps, Ms, Vs, Ws) for t in part if t is not None and t.numel()):
        raise ValueError("tensors of a plan must be 16-byte aligned (all but the exponents)")
    ptr = lambda t: _ptr(t).value if t is not None and t.numel() else None  # noqa: E731
    jobs = (AdamwJob * n)(*[
        AdamwJob(None, ptr(Ps[k]), ptr(Ms[k]), ptr(Vs[k]), ptr(M_exps[k]) if state8 else None,
                 ptr(V_exps[k]) if state8 else None, ptr(Ws[k]), sizes[k], lrs[k], decays[k]) for k in range(n)])
    return AdamwPlan(jobs, (list(Ps), list(Ms), list(Vs), list(Ws), *more), sizes, state8)


def sp24_adamw_step(plan, Gs, betas=(0.9, 0.999), eps=1e-8, step=None, control=None, seed=0, stream=None):
    """One AdamW step of a plan's tensors, in place, with the gradients ``Gs``
    (all float16 or all float32, each of its tensor's shape): the ``step``-th (1,
    2, ...), or as a control that sp24_grad_norm wrote says."""
    if (step is None) == (control is None):
        raise ValueError("either step or control")
    kind, pointers, sizes = _gradients(Gs)
    plan.check(Gs, sizes)
    if pointers and plan.tensors[0][0].get_device() != Gs[0].get_device():
        raise ValueError("the plan's tensors are not on the current device")
    plan.gradients[:] = pointers
    control = None if control is None else _addresses(_control(control))[0]
    _check("sp24_adamw_step", lib().sp24_adamw_step(
        plan.address, len(sizes), kind, STATE8 if plan.state8 else F32, float(betas[0]), float(betas[1]), float(eps),
        0 if step is None else int(step), control, int(seed) & 0xFFFFFFFF, _stream(stream)))


def state8(P):
    """An 8-bit state of zeros for a tensor: codes (uint8, P's shape) and
    exponents (uint8 [ceil(n / 64)])."""
    return (torch.zeros(P.shape, dtype=torch.uint8, device=P.device),
            torch.zeros(-(-P.numel() // 64), dtype=torch.uint8, device=P.device))


def sp24_state8_values(codes, exps, root=False, dtype=torch.float32, out=None, stream=None):
    """What an 8-bit state stands for, in codes' shape: M's entries, or with
    ``root`` the roots of V's; float32 or bfloat16 (which holds them whole)."""
    types = {torch.float32: F32, torch.bfloat16: BF16}
    if dtype not in types or codes.dtype != torch.uint8:
        raise ValueError("codes must be uint8, dtype float32 or bfloat16")
    _need(exps, (-(-codes.numel() // 64),), torch.uint8, "exps")
    with _using(stream):
        out = _out(out, codes.shape, dtype, codes.device)
    _check("sp24_state8_values", lib().sp24_state8_values(_ptr(codes), _ptr(exps), codes.numel(), int(bool(root)),
                                                          types[dtype], _ptr(out), _stream(stream)))
    return out
