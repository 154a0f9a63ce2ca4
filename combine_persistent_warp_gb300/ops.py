"""Operators around the expert layer: layer norm, the router with its gradient, rows into and
out of expert order, and products with one weight per expert over ragged groups of rows.

Entry points over the C ABI of include/cpw_moe.h; the module ``_ops`` (csrc/bind.cpp) marshals the
arguments.  Shapes, types and devices are checked there (``ValueError`` / ``TypeError``), sizes and
alignment by the library (:class:`MoeError`).  Every call is asynchronous on ``stream`` (default: the
current stream) and takes its outputs from PyTorch's pool of that stream; with another stream than
the current one, inputs are marked as in use there, and the caller orders the streams.  An ``out``
shares no memory with an input.

    h = ops.layer_norm(x, g, b)[0]
    idx, w = ops.route_topk(logits, topk)
    order = ops.expert_order(idx, E)
    rows = ops.gather_rows(h, order.rows, order.offsets)          # [T*topk, H], by expert
    y = ops.grouped_mm(rows, weights, order.offsets)              # weights [E, N, H]
    out = ops.combine_rows(y, order.rows, w)                      # [T, N]

``training`` has these as autograd functions.  The calls here are opaque to PyTorch: they record no
gradient, and cannot be traced, compiled or mapped.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import build, native
from .native import MoeError  # noqa: F401

native.load()
build.build_binding()
from . import _ops  # noqa: E402  (linked against the library, and like it built where it is missing)


class ExpertOrder(NamedTuple):
    """Expert-major order of a batch's (token, slot) pairs."""
    offsets: torch.Tensor   # int32 [E+1]: expert e has rows offsets[e] .. offsets[e+1]
    rows: torch.Tensor      # int32 [T, topk]: the row of each slot, -1 for a skipped one
    status: torch.Tensor    # int32 [1]: 0, or MOE_ERR_BAD_INDEX for an id outside [-1, E)


def _call(stream, fn, *args):
    """fn on another stream than the current one."""
    for t in args:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args)


# -------------------------------------------------------------------------- layer norm ----
def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, *, stream=None):
    """y = (x - mean) * rstd * weight + bias over the last dimension of x [T, H] (rows may be
    strided).  Returns (y, mean, rstd): y of x's type, mean and rstd fp32 [T]."""
    if stream is None:
        return _ops.layer_norm(x, weight, bias, eps)
    return _call(stream, _ops.layer_norm, x, weight, bias, eps)


def layer_norm_fp8(x, weight=None, bias=None, eps: float = 1e-5, *, pow2_scales: bool = False, stream=None):
    """Layer norm as FusedMoE.forward's activations: (e4m3 bytes uint8 [T, H], fp32 scales [T, H/128])."""
    if stream is None:
        return _ops.layer_norm_fp8(x, weight, bias, eps, pow2_scales)
    return _call(stream, _ops.layer_norm_fp8, x, weight, bias, eps, pow2_scales)


def layer_norm_backward(dy, x, weight, mean, rstd, *, param_dtype=None, weight_grad: bool = True, bias_grad: bool = True,
                        stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm.  dweight and dbias are of the weight's type
    (without a weight: ``param_dtype``, float32 or by default x's type); one that is not asked for is
    None, and without either their sums are not taken."""
    if param_dtype is not None and param_dtype != torch.float32 and param_dtype != x.dtype:
        raise TypeError(f"param_dtype: {param_dtype} is neither {x.dtype} nor float32")
    args = dy, x, weight, mean, rstd, param_dtype == torch.float32, weight_grad, bias_grad
    if stream is None:
        return _ops.layer_norm_backward(*args)
    return _call(stream, _ops.layer_norm_backward, *args)


# ------------------------------------------------------------------------------ router ----
def route_topk(logits, topk: int, *, token_mask=None, renormalize: bool = True, stream=None):
    """Top-k experts of each token and their gate weights, FusedMoE.forward's (topk_idx int64, topk_w
    fp32) [T, topk].  Ties go to the lowest expert; -inf logits and tokens whose ``token_mask`` (bool [T])
    is False choose nothing: idx -1, weight 0."""
    if stream is None:
        return _ops.route_topk(logits, topk, token_mask, renormalize)
    return _call(stream, _ops.route_topk, logits, topk, token_mask, renormalize)


def route_topk_backward(dw, idx, w, logits, *, renormalize: bool = True, stream=None):
    """Gradient of the logits (their type) from dw, that of the gate weights (fp32 [T, topk])."""
    if stream is None:
        return _ops.route_topk_backward(dw, idx, w, logits, renormalize)
    return _call(stream, _ops.route_topk_backward, dw, idx, w, logits, renormalize)


def expert_order(idx, E: int, *, stream=None) -> ExpertOrder:
    """Expert-major order of the slots idx [T, topk] names (-1: skipped): by expert, token, slot."""
    return ExpertOrder(*(_ops.expert_order(idx, E) if stream is None else _call(stream, _ops.expert_order, idx, E)))


# -------------------------------------------------------------------------------- rows ----
def gather_rows(x, rows, offsets, *, stream=None):
    """Rows of x [T, H] in expert order: out [T*topk, H] with out[rows[t, j]] = x[t], and zeros in the
    rows from offsets[E] on.  rows and offsets are an ``expert_order``, in which every row before has its
    slot: to skip a slot, put -1 into the order's idx, not into its rows.  Its gradient is
    ``combine_rows(dout, rows)``."""
    if stream is None:
        return _ops.gather_rows(x, rows, offsets)
    return _call(stream, _ops.gather_rows, x, rows, offsets)


def combine_rows(y, rows, w=None, *, stream=None):
    """out[t] = sum_j w[t, j] * y[rows[t, j]] (w fp32 [T, topk], None: ones) in fp32, rounded once."""
    if stream is None:
        return _ops.combine_rows(y, rows, w)
    return _call(stream, _ops.combine_rows, y, rows, w)


def combine_rows_backward(dout, y, rows, w, offsets, *, gate_grad: bool = True, stream=None):
    """Gradients (dy, dw) of combine_rows: dy like y, dw fp32 [T, topk] (None without ``gate_grad``).
    rows and offsets as in ``gather_rows``."""
    if stream is None:
        return _ops.combine_rows_backward(dout, y, rows, w, offsets, gate_grad)
    return _call(stream, _ops.combine_rows_backward, dout, y, rows, w, offsets, gate_grad)


# -------------------------------------------------------------------- grouped products ----
def grouped_mm(x, w, offsets, *, out=None, stream=None):
    """out[r] = w[e] @ x[r] for the rows r of each expert e: x [M, K], w [E, N, K], out [M, N]
    (bfloat16 or float16; rows of x and out may be strided).  Rows past offsets[E] give zeros."""
    if stream is None:
        return _ops.grouped_mm(x, w, offsets, out)
    return _call(stream, _ops.grouped_mm, x, w, offsets, out)


def grouped_mm_dx(dy, w, offsets, *, out=None, stream=None):
    """Gradient of grouped_mm's x: out[r] = dy[r] @ w[e], dy [M, N], w [E, N, K], out [M, K]."""
    if stream is None:
        return _ops.grouped_mm_dx(dy, w, offsets, out)
    return _call(stream, _ops.grouped_mm_dx, dy, w, offsets, out)


def grouped_mm_dw(dy, x, offsets, *, out=None, accumulate: bool = False, dtype=None, stream=None):
    """Gradient of grouped_mm's w: out[e] = dy[rows of e]^T @ x[rows of e], dy [M, N], x [M, K],
    out [E, N, K] of x's type or (``dtype``) float32; with ``accumulate`` added to ``out``."""
    want = dtype if dtype is not None else x.dtype if out is None else out.dtype
    if want != torch.float32 and want != x.dtype:
        raise TypeError(f"out: dtype {want} is neither {x.dtype} nor float32")
    if out is not None and out.dtype != want:
        raise TypeError(f"out: dtype {out.dtype} != {want}")
    if stream is None:
        return _ops.grouped_mm_dw(dy, x, offsets, out, accumulate, want == torch.float32)
    return _call(stream, _ops.grouped_mm_dw, dy, x, offsets, out, accumulate, want == torch.float32)


def get_error(stream=None) -> int:
    """Waits for ``stream`` (default: the current stream), then returns (and clears) the sticky status
    of the grouped products' bounded waits: 0 or MOE_ERR_TIMEOUT.  After the latter what they wrote is
    undefined.  The status is the device's: one that another thread asked for is cleared."""
    if stream is None:
        return _ops.get_error()
    return _call(stream, _ops.get_error)
