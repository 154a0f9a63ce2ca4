"""Operators around the expert layer: layer norm, the router with its gradient, rows into and
out of expert order, and products with one weight per expert over ragged groups of rows.

Argument marshalling over the C ABI of include/cpw_moe.h, as in ``native``: shapes, types and
devices are checked here (``ValueError`` / ``TypeError``), sizes and alignment by the library
(:class:`MoeError`).  Every call is asynchronous on ``stream`` (default: the current stream) and
allocates its outputs from PyTorch's pool of that stream; with another stream than the current one, inputs are
marked as in use there, and the caller orders the streams.

    h = ops.layer_norm(x, g, b)[0]
    idx, w = ops.route_topk(logits, topk)
    order = ops.expert_order(idx, E)
    rows = ops.gather_rows(h, order.rows, order.offsets)          # [T*topk, H], by expert
    y = ops.grouped_mm(rows, weights, order.offsets)              # weights [E, N, H]
    out = ops.combine_rows(y, order.rows, w)                      # [T, N]

``training`` has these as autograd functions.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import native
from .native import MoeError, _check  # noqa: F401

_DTYPE = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}


class ExpertOrder(NamedTuple):
    """Expert-major order of a batch's (token, slot) pairs."""
    offsets: torch.Tensor   # int32 [E+1]: expert e has rows offsets[e] .. offsets[e+1]
    rows: torch.Tensor      # int32 [T, topk]: the row of each slot, -1 for a skipped one
    status: torch.Tensor    # int32 [1]: 0, or MOE_ERR_BAD_INDEX for an id outside [-1, E)


# ------------------------------------------------------------------------- marshalling ----
def _dtype(t, name):
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16") from None


def _rows(t, name, width=None, like=None, dtype=None):
    """A CUDA matrix of contiguous rows; returns its row stride in elements."""
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not [rows, {width if width is not None else 'width'}]")
    _device(t, name, like)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    n, w = t.shape
    if n <= 1:
        if w > 1 and n == 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        return max(w, 1) if n == 0 or t.stride(0) < w else t.stride(0)
    if (w > 1 and t.stride(1) != 1) or t.stride(0) < w:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return t.stride(0)


def _flat(t, name, shape, dtype, like=None):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _device(t, name, like)


def _device(t, name, like):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if like is not None:
        if t.device != like.device:
            raise ValueError(f"{name} is on {t.device}, other tensors on {like.device}")
    elif t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")


def _affine(t, name, width, like):
    """A weight or bias [H] of x's type or fp32 (or None): its pointer."""
    if t is None:
        return None
    if t.dtype != like.dtype and t.dtype != torch.float32:
        raise TypeError(f"{name}: dtype {t.dtype} is neither {like.dtype} nor float32")
    _flat(t, name, (width,), t.dtype, like)
    return t.data_ptr()


def _affine_dtype(x, *params):
    kinds = {p.dtype for p in params if p is not None}
    if len(kinds) > 1:
        raise TypeError("weight and bias must have one dtype")
    return _DTYPE[kinds.pop()] if kinds else _DTYPE[x.dtype]


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream(stream, *inputs):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _out(out, name, shape, dtype, like, stream):
    """The caller's output matrix (rows may be strided) or a new one, and its row stride."""
    if out is None:
        return _empty(shape, dtype, like.device, stream), max(shape[1], 1)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(out.shape)} != {tuple(shape)}")
    return out, _rows(out, name, like=like, dtype=dtype)


# -------------------------------------------------------------------------- layer norm ----
def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, stream=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension of x [T, H] (rows may be
    strided).  Returns (y, mean, rstd): y of x's type, mean and rstd fp32 [T]."""
    ldx, dt = _rows(x, "x"), _dtype(x, "x")
    T, H = x.shape
    w, b = _affine(weight, "weight", H, x), _affine(bias, "bias", H, x)
    wdt = _affine_dtype(x, weight, bias)
    y = _empty((T, H), x.dtype, x.device, stream)
    mean = _empty((T,), torch.float32, x.device, stream)
    rstd = _empty((T,), torch.float32, x.device, stream)
    _check(native.load().moe_layer_norm(T, H, x.data_ptr(), ldx, dt, w, b, wdt, eps, y.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), _stream(stream, x, weight, bias)), "moe_layer_norm")
    return y, mean, rstd


def layer_norm_fp8(x, weight=None, bias=None, eps: float = 1e-5, *, pow2_scales: bool = False, stream=None):
    """Layer norm as FusedMoE.forward's activations: (e4m3 bytes uint8 [T, H], fp32 scales [T, H/128])."""
    ldx, dt = _rows(x, "x"), _dtype(x, "x")
    T, H = x.shape
    w, b = _affine(weight, "weight", H, x), _affine(bias, "bias", H, x)
    wdt = _affine_dtype(x, weight, bias)
    q = _empty((T, H), torch.uint8, x.device, stream)
    sf = _empty((T, H // 128), torch.float32, x.device, stream)
    _check(native.load().moe_layer_norm_fp8(T, H, x.data_ptr(), ldx, dt, w, b, wdt, eps, int(pow2_scales), q.data_ptr(),
                                            sf.data_ptr(), _stream(stream, x, weight, bias)), "moe_layer_norm_fp8")
    return q, sf


def layer_norm_backward(dy, x, weight, mean, rstd, *, param_dtype=None, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm.  dweight and dbias are of the weight's type
    (without a weight: ``param_dtype``, by default x's)."""
    ldx, dt = _rows(x, "x"), _dtype(x, "x")
    T, H = x.shape
    lddy = _rows(dy, "dy", H, like=x, dtype=x.dtype)
    if dy.shape[0] != T:
        raise ValueError(f"dy: {dy.shape[0]} rows, x has {T}")
    w = _affine(weight, "weight", H, x)
    _flat(mean, "mean", (T,), torch.float32, x)
    _flat(rstd, "rstd", (T,), torch.float32, x)
    pdt = weight.dtype if weight is not None else (param_dtype or x.dtype)
    if pdt not in (x.dtype, torch.float32):
        raise TypeError(f"param_dtype: {pdt} is neither {x.dtype} nor float32")
    L = native.load()
    need = ctypes.c_uint64()
    _check(L.moe_layer_norm_backward_workspace(T, H, ctypes.byref(need)), "moe_layer_norm_backward_workspace")
    ws = _empty((need.value,), torch.uint8, x.device, stream)
    dx = _empty((T, H), x.dtype, x.device, stream)
    dweight = _empty((H,), pdt, x.device, stream)
    dbias = _empty((H,), pdt, x.device, stream)
    _check(L.moe_layer_norm_backward(T, H, dy.data_ptr(), lddy, x.data_ptr(), ldx, dt, w, _DTYPE[pdt], mean.data_ptr(),
                                     rstd.data_ptr(), dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), ws.data_ptr(),
                                     need.value, _stream(stream, dy, x, weight, mean, rstd)), "moe_layer_norm_backward")
    return dx, dweight, dbias


# ------------------------------------------------------------------------------ router ----
def route_topk(logits, topk: int, *, token_mask=None, renormalize: bool = True, stream=None):
    """Top-k experts of each token and their gate weights, FusedMoE.forward's (topk_idx int64, topk_w
    fp32) [T, topk].  Ties go to the lowest expert; -inf logits and tokens whose ``token_mask`` (bool [T])
    is False choose nothing: idx -1, weight 0."""
    ld, dt = _rows(logits, "logits"), _dtype(logits, "logits")
    T, E = logits.shape
    if token_mask is not None:
        _flat(token_mask, "token_mask", (T,), torch.bool, logits)
    idx = _empty((T, topk), torch.int64, logits.device, stream)
    w = _empty((T, topk), torch.float32, logits.device, stream)
    _check(native.load().moe_route_topk(T, E, topk, logits.data_ptr(), ld, dt, _ptr(token_mask), int(renormalize),
                                        idx.data_ptr(), w.data_ptr(), _stream(stream, logits, token_mask)),
           "moe_route_topk")
    return idx, w


def route_topk_backward(dw, idx, w, logits, *, renormalize: bool = True, stream=None):
    """Gradient of the logits (their type) from dw, that of the gate weights (fp32 [T, topk])."""
    ld, dt = _rows(logits, "logits"), _dtype(logits, "logits")
    T, E = logits.shape
    if idx.dim() != 2:
        raise ValueError(f"idx: shape {tuple(idx.shape)} is not [T, topk]")
    k = idx.shape[1]
    _flat(idx, "idx", (T, k), torch.int64, logits)
    _flat(w, "w", (T, k), torch.float32, logits)
    _flat(dw, "dw", (T, k), torch.float32, logits)
    d = _empty((T, E), logits.dtype, logits.device, stream)
    _check(native.load().moe_route_topk_backward(T, E, k, dw.data_ptr(), idx.data_ptr(), w.data_ptr(), logits.data_ptr(),
                                                 ld, dt, int(renormalize), d.data_ptr(),
                                                 _stream(stream, dw, idx, w, logits)), "moe_route_topk_backward")
    return d


def expert_order(idx, E: int, *, stream=None) -> ExpertOrder:
    """Expert-major order of the slots idx [T, topk] names (-1: skipped): by expert, token, slot."""
    if idx.dim() != 2:
        raise ValueError(f"idx: shape {tuple(idx.shape)} is not [T, topk]")
    T, k = idx.shape
    _flat(idx, "idx", (T, k), torch.int64)
    L = native.load()
    need = ctypes.c_uint64()
    _check(L.moe_expert_order_workspace(T, k, E, ctypes.byref(need)), "moe_expert_order_workspace")
    ws = _empty((need.value,), torch.uint8, idx.device, stream) if need.value else None
    offsets = _empty((E + 1,), torch.int32, idx.device, stream)
    rows = _empty((T, k), torch.int32, idx.device, stream)
    status = _empty((1,), torch.int32, idx.device, stream)
    _check(L.moe_expert_order(T, k, E, idx.data_ptr(), offsets.data_ptr(), rows.data_ptr(), status.data_ptr(), _ptr(ws),
                              need.value, _stream(stream, idx)), "moe_expert_order")
    return ExpertOrder(offsets, rows, status)


# -------------------------------------------------------------------------------- rows ----
def _order_args(rows, offsets, like):
    if rows.dim() != 2:
        raise ValueError(f"rows: shape {tuple(rows.shape)} is not [T, topk]")
    _flat(rows, "rows", rows.shape, torch.int32, like)
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError(f"offsets: shape {tuple(offsets.shape)} is not [E+1]")
        _flat(offsets, "offsets", offsets.shape, torch.int32, like)
    return rows.shape


def gather_rows(x, rows, offsets, *, stream=None):
    """Rows of x [T, H] in expert order: out [T*topk, H] with out[rows[t, j]] = x[t], and zeros in the
    rows that no slot has.  Its gradient is ``combine_rows(dout, rows)``."""
    ldx, dt = _rows(x, "x"), _dtype(x, "x")
    T, k = _order_args(rows, offsets, x)
    if x.shape[0] != T:
        raise ValueError(f"x: {x.shape[0]} rows, rows has {T}")
    H = x.shape[1]
    out = _empty((T * k, H), x.dtype, x.device, stream)
    _check(native.load().moe_gather_rows(T, k, H, offsets.shape[0] - 1, T * k, x.data_ptr(), ldx, dt, rows.data_ptr(),
                                         offsets.data_ptr(), out.data_ptr(), _stream(stream, x, rows, offsets)),
           "moe_gather_rows")
    return out


def combine_rows(y, rows, w=None, *, stream=None):
    """out[t] = sum_j w[t, j] * y[rows[t, j]] (w fp32 [T, topk], None: ones) in fp32, rounded once."""
    dt = _dtype(y, "y")
    if y.dim() != 2:
        raise ValueError(f"y: shape {tuple(y.shape)} is not [rows, H]")
    M, H = y.shape
    _flat(y, "y", (M, H), y.dtype)
    T, k = _order_args(rows, None, y)
    if w is not None:
        _flat(w, "w", (T, k), torch.float32, y)
    out = _empty((T, H), y.dtype, y.device, stream)
    _check(native.load().moe_combine_rows(T, k, H, M, y.data_ptr(), dt, rows.data_ptr(), _ptr(w), out.data_ptr(),
                                          _stream(stream, y, rows, w)), "moe_combine_rows")
    return out


def combine_rows_backward(dout, y, rows, w, offsets, *, stream=None):
    """Gradients (dy, dw) of combine_rows: dy like y, dw fp32 [T, topk]."""
    dt = _dtype(y, "y")
    if y.dim() != 2:
        raise ValueError(f"y: shape {tuple(y.shape)} is not [rows, H]")
    M, H = y.shape
    _flat(y, "y", (M, H), y.dtype)
    T, k = _order_args(rows, offsets, y)
    ld = _rows(dout, "dout", H, like=y, dtype=y.dtype)
    if dout.shape[0] != T:
        raise ValueError(f"dout: {dout.shape[0]} rows, rows has {T}")
    if w is not None:
        _flat(w, "w", (T, k), torch.float32, y)
    dy = _empty((M, H), y.dtype, y.device, stream)
    dw = _empty((T, k), torch.float32, y.device, stream)
    _check(native.load().moe_combine_rows_backward(T, k, H, offsets.shape[0] - 1, M, dout.data_ptr(), ld, y.data_ptr(), dt,
                                                   rows.data_ptr(), _ptr(w), offsets.data_ptr(), dy.data_ptr(),
                                                   dw.data_ptr(), _stream(stream, dout, y, rows, w, offsets)),
           "moe_combine_rows_backward")
    return dy, dw


# -------------------------------------------------------------------- grouped products ----
def _weights(w, dtype, like):
    if w.dim() != 3:
        raise ValueError(f"w: shape {tuple(w.shape)} is not [E, N, K]")
    _flat(w, "w", w.shape, dtype, like)
    return w.shape


def _half(t, name):
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name}: dtype {t.dtype} is not bfloat16 or float16")
    return _DTYPE[t.dtype]


def _offsets(offsets, E, like):
    _flat(offsets, "offsets", (E + 1,), torch.int32, like)


def grouped_mm(x, w, offsets, *, out=None, stream=None):
    """out[r] = w[e] @ x[r] for the rows r of each expert e: x [M, K], w [E, N, K], out [M, N]
    (bfloat16 or float16; rows of x and out may be strided).  Rows past offsets[E] give zeros."""
    dt = _half(x, "x")
    E, N, K = _weights(w, x.dtype, x)
    ldx = _rows(x, "x", K)
    _offsets(offsets, E, x)
    out, ldo = _out(out, "out", (x.shape[0], N), x.dtype, x, stream)
    _check(native.load().moe_grouped_mm(x.shape[0], E, N, K, x.data_ptr(), ldx, w.data_ptr(), offsets.data_ptr(),
                                        out.data_ptr(), ldo, dt, _stream(stream, x, w, offsets)), "moe_grouped_mm")
    return out


def grouped_mm_dx(dy, w, offsets, *, out=None, stream=None):
    """Gradient of grouped_mm's x: out[r] = dy[r] @ w[e], dy [M, N], w [E, N, K], out [M, K]."""
    dt = _half(dy, "dy")
    E, N, K = _weights(w, dy.dtype, dy)
    lddy = _rows(dy, "dy", N)
    _offsets(offsets, E, dy)
    out, ldo = _out(out, "out", (dy.shape[0], K), dy.dtype, dy, stream)
    _check(native.load().moe_grouped_mm_dx(dy.shape[0], E, N, K, dy.data_ptr(), lddy, w.data_ptr(), offsets.data_ptr(),
                                           out.data_ptr(), ldo, dt, _stream(stream, dy, w, offsets)), "moe_grouped_mm_dx")
    return out


def grouped_mm_dw(dy, x, offsets, *, out=None, accumulate: bool = False, dtype=None, stream=None):
    """Gradient of grouped_mm's w: out[e] = dy[rows of e]^T @ x[rows of e], dy [M, N], x [M, K],
    out [E, N, K] of x's type or (``dtype``) float32; with ``accumulate`` added to ``out``."""
    dt = _half(x, "x")
    ldx = _rows(x, "x")
    M, K = x.shape
    lddy = _rows(dy, "dy", like=x, dtype=x.dtype)
    if dy.shape[0] != M:
        raise ValueError(f"dy: {dy.shape[0]} rows, x has {M}")
    N = dy.shape[1]
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets: shape {tuple(offsets.shape)} is not [E+1]")
    E = offsets.shape[0] - 1
    _offsets(offsets, E, x)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out to add to")
        out = _empty((E, N, K), dtype or x.dtype, x.device, stream)
    else:
        _flat(out, "out", (E, N, K), dtype or out.dtype, x)
    if out.dtype not in (x.dtype, torch.float32):
        raise TypeError(f"out: dtype {out.dtype} is neither {x.dtype} nor float32")
    L = native.load()
    need = ctypes.c_uint64()
    _check(L.moe_grouped_mm_dw_workspace(E, ctypes.byref(need)), "moe_grouped_mm_dw_workspace")
    ws = _empty((need.value,), torch.uint8, x.device, stream)
    _check(L.moe_grouped_mm_dw(M, E, N, K, dy.data_ptr(), lddy, x.data_ptr(), ldx, offsets.data_ptr(), out.data_ptr(), dt,
                               _DTYPE[out.dtype], int(accumulate), ws.data_ptr(), need.value,
                               _stream(stream, dy, x, offsets)), "moe_grouped_mm_dw")
    return out


def get_error(stream=None) -> int:
    """Waits for ``stream``, then returns (and clears) the sticky status of the grouped products'
    bounded waits: 0 or MOE_ERR_TIMEOUT."""
    st = ctypes.c_int(0)
    _check(native.load().moe_ops_get_error(ctypes.byref(st), _stream(stream)), "moe_ops_get_error")
    return st.value
