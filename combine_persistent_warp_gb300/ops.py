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
import functools
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
# These calls are a few microseconds of GPU work at decode sizes, so the checks are kept to one
# look at each property of a tensor.
def _bad(t, name, dtype):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype} != {dtype}")
    raise ValueError(f"{name} is on {t.device}, not on the current device or other tensors' device")


def _first(t, name):
    """Element type and device of the matrix that the other tensors are held against."""
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not [rows, width]")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16")
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _bad(t, name, None)
    return code, dev


def _rows(t, name, dtype, dev, rows=None, width=None):
    """A matrix of contiguous rows: its shape and row stride in elements."""
    shape = t.shape
    if len(shape) != 2 or (width is not None and shape[1] != width) or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: shape {tuple(shape)} is not [{'rows' if rows is None else rows}, {'width' if width is None else width}]")
    if t.dtype != dtype or t.get_device() != dev:
        _bad(t, name, dtype)
    n, w = shape
    ld, step = t.stride()
    if n <= 1:
        if n == 1 and w > 1 and step != 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        return n, w, max(ld, w, 1)
    if (w > 1 and step != 1) or ld < w:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return n, w, ld


def _flat(t, name, shape, dtype, dev):
    """A contiguous tensor of the given shape: its address."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype or t.get_device() != dev:
        _bad(t, name, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _affine(weight, bias, width, dtype, dev):
    """A norm's weight and bias [H] (or None), both of x's type or both fp32: addresses and type."""
    kind = dtype if weight is None and bias is None else (weight if weight is not None else bias).dtype
    if kind != dtype and kind != torch.float32:
        raise TypeError(f"weight and bias: dtype {kind} is neither {dtype} nor float32")
    return (None if weight is None else _flat(weight, "weight", (width,), kind, dev),
            None if bias is None else _flat(bias, "bias", (width,), kind, dev), _DTYPE[kind])


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream(stream, dev, *inputs):
    if stream is None:
        return _current_stream(dev)
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _current_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(call, dev, *sizes):
    """Bytes of a call's workspace, which depend on the sizes and the kind of GPU alone."""
    need = ctypes.c_uint64()
    _check(getattr(native.load(), call)(*sizes, ctypes.byref(need)), call)
    return need.value


def _workspace(call, dev, device, stream, *sizes):
    """A workspace of this stream (address and bytes; kept alive by the first item)."""
    need = _workspace_bytes(call, dev, *sizes)
    if need == 0:
        return None, None, 0
    t = _empty((need,), torch.uint8, device, stream)
    return t, t.data_ptr(), need


# -------------------------------------------------------------------------- layer norm ----
def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, stream=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension of x [T, H] (rows may be
    strided).  Returns (y, mean, rstd): y of x's type, mean and rstd fp32 [T]."""
    dt, dev = _first(x, "x")
    T, H, ldx = _rows(x, "x", x.dtype, dev)
    w, b, wdt = _affine(weight, bias, H, x.dtype, dev)
    device = x.device
    y = _empty((T, H), x.dtype, device, stream)
    mean = _empty((T,), torch.float32, device, stream)
    rstd = _empty((T,), torch.float32, device, stream)
    rc = native.load().moe_layer_norm(T, H, x.data_ptr(), ldx, dt, w, b, wdt, eps, y.data_ptr(), mean.data_ptr(),
                                      rstd.data_ptr(), _stream(stream, dev, x, weight, bias))
    if rc:
        _check(rc, "moe_layer_norm")
    return y, mean, rstd


def layer_norm_fp8(x, weight=None, bias=None, eps: float = 1e-5, *, pow2_scales: bool = False, stream=None):
    """Layer norm as FusedMoE.forward's activations: (e4m3 bytes uint8 [T, H], fp32 scales [T, H/128])."""
    dt, dev = _first(x, "x")
    T, H, ldx = _rows(x, "x", x.dtype, dev)
    w, b, wdt = _affine(weight, bias, H, x.dtype, dev)
    device = x.device
    q = _empty((T, H), torch.uint8, device, stream)
    sf = _empty((T, H // 128), torch.float32, device, stream)
    rc = native.load().moe_layer_norm_fp8(T, H, x.data_ptr(), ldx, dt, w, b, wdt, eps, int(pow2_scales), q.data_ptr(),
                                          sf.data_ptr(), _stream(stream, dev, x, weight, bias))
    if rc:
        _check(rc, "moe_layer_norm_fp8")
    return q, sf


def layer_norm_backward(dy, x, weight, mean, rstd, *, param_dtype=None, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm.  dweight and dbias are of the weight's type
    (without a weight: ``param_dtype``, by default x's)."""
    dt, dev = _first(x, "x")
    T, H, ldx = _rows(x, "x", x.dtype, dev)
    _, _, lddy = _rows(dy, "dy", x.dtype, dev, T, H)
    w, _, wdt = _affine(weight, None, H, x.dtype, dev)
    pm, pr = _flat(mean, "mean", (T,), torch.float32, dev), _flat(rstd, "rstd", (T,), torch.float32, dev)
    pdt = weight.dtype if weight is not None else (param_dtype or x.dtype)
    if pdt != x.dtype and pdt != torch.float32:
        raise TypeError(f"param_dtype: {pdt} is neither {x.dtype} nor float32")
    L, device = native.load(), x.device
    ws, pws, need = _workspace("moe_layer_norm_backward_workspace", dev, device, stream, T, H)
    dx = _empty((T, H), x.dtype, device, stream)
    dweight = _empty((H,), pdt, device, stream)
    dbias = _empty((H,), pdt, device, stream)
    rc = L.moe_layer_norm_backward(T, H, dy.data_ptr(), lddy, x.data_ptr(), ldx, dt, w, _DTYPE[pdt], pm, pr, dx.data_ptr(),
                                   dweight.data_ptr(), dbias.data_ptr(), pws, need,
                                   _stream(stream, dev, dy, x, weight, mean, rstd))
    if rc:
        _check(rc, "moe_layer_norm_backward")
    return dx, dweight, dbias


# ------------------------------------------------------------------------------ router ----
def route_topk(logits, topk: int, *, token_mask=None, renormalize: bool = True, stream=None):
    """Top-k experts of each token and their gate weights, FusedMoE.forward's (topk_idx int64, topk_w
    fp32) [T, topk].  Ties go to the lowest expert; -inf logits and tokens whose ``token_mask`` (bool [T])
    is False choose nothing: idx -1, weight 0."""
    dt, dev = _first(logits, "logits")
    T, E, ld = _rows(logits, "logits", logits.dtype, dev)
    mask = None if token_mask is None else _flat(token_mask, "token_mask", (T,), torch.bool, dev)
    device = logits.device
    idx = _empty((T, topk), torch.int64, device, stream)
    w = _empty((T, topk), torch.float32, device, stream)
    rc = native.load().moe_route_topk(T, E, topk, logits.data_ptr(), ld, dt, mask, int(renormalize), idx.data_ptr(),
                                      w.data_ptr(), _stream(stream, dev, logits, token_mask))
    if rc:
        _check(rc, "moe_route_topk")
    return idx, w


def _slots(idx):
    if idx.dim() != 2:
        raise ValueError(f"idx: shape {tuple(idx.shape)} is not [T, topk]")
    return idx.shape


def route_topk_backward(dw, idx, w, logits, *, renormalize: bool = True, stream=None):
    """Gradient of the logits (their type) from dw, that of the gate weights (fp32 [T, topk])."""
    dt, dev = _first(logits, "logits")
    T, E, ld = _rows(logits, "logits", logits.dtype, dev)
    k = _slots(idx)[1]
    pi = _flat(idx, "idx", (T, k), torch.int64, dev)
    pw, pd = _flat(w, "w", (T, k), torch.float32, dev), _flat(dw, "dw", (T, k), torch.float32, dev)
    d = _empty((T, E), logits.dtype, logits.device, stream)
    rc = native.load().moe_route_topk_backward(T, E, k, pd, pi, pw, logits.data_ptr(), ld, dt, int(renormalize), d.data_ptr(),
                                               _stream(stream, dev, dw, idx, w, logits))
    if rc:
        _check(rc, "moe_route_topk_backward")
    return d


def expert_order(idx, E: int, *, stream=None) -> ExpertOrder:
    """Expert-major order of the slots idx [T, topk] names (-1: skipped): by expert, token, slot."""
    T, k = _slots(idx)
    dev = idx.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _bad(idx, "idx", torch.int64)
    pi = _flat(idx, "idx", (T, k), torch.int64, dev)
    L, device = native.load(), idx.device
    ws, pws, need = _workspace("moe_expert_order_workspace", dev, device, stream, T, k, E)
    offsets = _empty((E + 1,), torch.int32, device, stream)
    rows = _empty((T, k), torch.int32, device, stream)
    status = _empty((1,), torch.int32, device, stream)
    rc = L.moe_expert_order(T, k, E, pi, offsets.data_ptr(), rows.data_ptr(), status.data_ptr(),
                            pws, need, _stream(stream, dev, idx))
    if rc:
        _check(rc, "moe_expert_order")
    return ExpertOrder(offsets, rows, status)


# -------------------------------------------------------------------------------- rows ----
def _order_rows(rows, dev):
    shape = rows.shape
    if len(shape) != 2:
        raise ValueError(f"rows: shape {tuple(shape)} is not [T, topk]")
    return shape[0], shape[1], _flat(rows, "rows", shape, torch.int32, dev)


def _groups(offsets, dev, E=None):
    shape = offsets.shape
    if len(shape) != 1 or shape[0] < 2 or (E is not None and shape[0] != E + 1):
        raise ValueError(f"offsets: shape {tuple(shape)} is not [{'E' if E is None else E}+1]")
    return shape[0] - 1, _flat(offsets, "offsets", shape, torch.int32, dev)


def gather_rows(x, rows, offsets, *, stream=None):
    """Rows of x [T, H] in expert order: out [T*topk, H] with out[rows[t, j]] = x[t], and zeros in the
    rows that no slot has.  Its gradient is ``combine_rows(dout, rows)``."""
    dt, dev = _first(x, "x")
    T, k, pr = _order_rows(rows, dev)
    _, H, ldx = _rows(x, "x", x.dtype, dev, T)
    E, po = _groups(offsets, dev)
    out = _empty((T * k, H), x.dtype, x.device, stream)
    rc = native.load().moe_gather_rows(T, k, H, E, T * k, x.data_ptr(), ldx, dt, pr, po, out.data_ptr(),
                                       _stream(stream, dev, x, rows, offsets))
    if rc:
        _check(rc, "moe_gather_rows")
    return out


def _matrix(y, dev):
    M, H = y.shape
    return M, H, _flat(y, "y", (M, H), y.dtype, dev)


def combine_rows(y, rows, w=None, *, stream=None):
    """out[t] = sum_j w[t, j] * y[rows[t, j]] (w fp32 [T, topk], None: ones) in fp32, rounded once."""
    dt, dev = _first(y, "y")
    M, H, py = _matrix(y, dev)
    T, k, pr = _order_rows(rows, dev)
    pw = None if w is None else _flat(w, "w", (T, k), torch.float32, dev)
    out = _empty((T, H), y.dtype, y.device, stream)
    rc = native.load().moe_combine_rows(T, k, H, M, py, dt, pr, pw, out.data_ptr(), _stream(stream, dev, y, rows, w))
    if rc:
        _check(rc, "moe_combine_rows")
    return out


def combine_rows_backward(dout, y, rows, w, offsets, *, stream=None):
    """Gradients (dy, dw) of combine_rows: dy like y, dw fp32 [T, topk]."""
    dt, dev = _first(y, "y")
    M, H, py = _matrix(y, dev)
    T, k, pr = _order_rows(rows, dev)
    E, po = _groups(offsets, dev)
    _, _, ld = _rows(dout, "dout", y.dtype, dev, T, H)
    pw = None if w is None else _flat(w, "w", (T, k), torch.float32, dev)
    dy = _empty((M, H), y.dtype, y.device, stream)
    dw = _empty((T, k), torch.float32, y.device, stream)
    rc = native.load().moe_combine_rows_backward(T, k, H, E, M, dout.data_ptr(), ld, py, dt, pr, pw, po, dy.data_ptr(),
                                                 dw.data_ptr(), _stream(stream, dev, dout, y, rows, w, offsets))
    if rc:
        _check(rc, "moe_combine_rows_backward")
    return dy, dw


# -------------------------------------------------------------------- grouped products ----
def _half(t, name):
    if t.dtype != torch.bfloat16 and t.dtype != torch.float16:
        raise TypeError(f"{name}: dtype {t.dtype} is not bfloat16 or float16")
    return _first(t, name)


def _weights(w, dtype, dev):
    shape = w.shape
    if len(shape) != 3:
        raise ValueError(f"w: shape {tuple(shape)} is not [E, N, K]")
    return (*shape, _flat(w, "w", shape, dtype, dev))


def _out(out, shape, dtype, device, dev, stream):
    """The caller's output matrix (rows may be strided) or a new one, and its row stride."""
    if out is None:
        return _empty(shape, dtype, device, stream), max(shape[1], 1)
    return out, _rows(out, "out", dtype, dev, *shape)[2]


def grouped_mm(x, w, offsets, *, out=None, stream=None):
    """out[r] = w[e] @ x[r] for the rows r of each expert e: x [M, K], w [E, N, K], out [M, N]
    (bfloat16 or float16; rows of x and out may be strided).  Rows past offsets[E] give zeros."""
    dt, dev = _half(x, "x")
    E, N, K, pw = _weights(w, x.dtype, dev)
    M, _, ldx = _rows(x, "x", x.dtype, dev, None, K)
    _, po = _groups(offsets, dev, E)
    out, ldo = _out(out, (M, N), x.dtype, x.device, dev, stream)
    rc = native.load().moe_grouped_mm(M, E, N, K, x.data_ptr(), ldx, pw, po, out.data_ptr(), ldo, dt,
                                      _stream(stream, dev, x, w, offsets))
    if rc:
        _check(rc, "moe_grouped_mm")
    return out


def grouped_mm_dx(dy, w, offsets, *, out=None, stream=None):
    """Gradient of grouped_mm's x: out[r] = dy[r] @ w[e], dy [M, N], w [E, N, K], out [M, K]."""
    dt, dev = _half(dy, "dy")
    E, N, K, pw = _weights(w, dy.dtype, dev)
    M, _, lddy = _rows(dy, "dy", dy.dtype, dev, None, N)
    _, po = _groups(offsets, dev, E)
    out, ldo = _out(out, (M, K), dy.dtype, dy.device, dev, stream)
    rc = native.load().moe_grouped_mm_dx(M, E, N, K, dy.data_ptr(), lddy, pw, po, out.data_ptr(), ldo, dt,
                                         _stream(stream, dev, dy, w, offsets))
    if rc:
        _check(rc, "moe_grouped_mm_dx")
    return out


def grouped_mm_dw(dy, x, offsets, *, out=None, accumulate: bool = False, dtype=None, stream=None):
    """Gradient of grouped_mm's w: out[e] = dy[rows of e]^T @ x[rows of e], dy [M, N], x [M, K],
    out [E, N, K] of x's type or (``dtype``) float32; with ``accumulate`` added to ``out``."""
    dt, dev = _half(x, "x")
    M, K, ldx = _rows(x, "x", x.dtype, dev)
    _, N, lddy = _rows(dy, "dy", x.dtype, dev, M)
    E, po = _groups(offsets, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an out to add to")
        out = _empty((E, N, K), dtype or x.dtype, x.device, stream)
    else:
        _flat(out, "out", (E, N, K), dtype or out.dtype, dev)
    if out.dtype != x.dtype and out.dtype != torch.float32:
        raise TypeError(f"out: dtype {out.dtype} is neither {x.dtype} nor float32")
    L = native.load()
    ws, pws, need = _workspace("moe_grouped_mm_dw_workspace", dev, x.device, stream, E)
    rc = L.moe_grouped_mm_dw(M, E, N, K, dy.data_ptr(), lddy, x.data_ptr(), ldx, po, out.data_ptr(), dt, _DTYPE[out.dtype],
                             int(accumulate), pws, need, _stream(stream, dev, dy, x, offsets))
    if rc:
        _check(rc, "moe_grouped_mm_dw")
    return out


def get_error(stream=None) -> int:
    """Waits for ``stream``, then returns (and clears) the sticky status of the grouped products'
    bounded waits: 0 or MOE_ERR_TIMEOUT."""
    st = ctypes.c_int(0)
    _check(native.load().moe_ops_get_error(ctypes.byref(st), _stream(stream, torch.cuda.current_device())),
           "moe_ops_get_error")
    return st.value
