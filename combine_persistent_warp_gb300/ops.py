"""Operators around the expert layer: layer and RMS norm, routers with their gradients, rows into and
out of expert order, products with one weight per expert over ragged groups of rows, the experts'
activation, and rows kept in 8 bits for the backward pass.

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

    h, rstd, x = ops.rms_norm(out, g, residual=x)                 # the stream goes on as x
    idx, w = ops.route_scores(logits, topk, bias=bias, groups=8, topk_groups=4)
    act, codes, scales = ops.swiglu_checkpoint(gate_up)           # codes and scales instead of gate_up

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


# ---------------------------------------------------------------------------- RMS norm ----
def rms_norm(x, weight=None, eps: float = 1e-6, *, residual=None, stream=None):
    """y = h * rstd * weight over the last dimension, rstd = 1 / sqrt(mean(h^2) + eps), of h = x + residual
    (both [T, H], of one type, in which the sum is kept; rows may be strided).  Returns (y, rstd, h): y and h of
    x's type, rstd fp32 [T]; without a residual h is x itself."""
    if stream is None:
        return _ops.rms_norm(x, weight, eps, residual)
    return _call(stream, _ops.rms_norm, x, weight, eps, residual)


def rms_norm_fp8(x, weight=None, eps: float = 1e-6, *, residual=None, pow2_scales: bool = False, stream=None):
    """RMS norm as FusedMoE.forward's activations: (e4m3 bytes uint8 [T, H], fp32 scales [T, H/128], h)."""
    if stream is None:
        return _ops.rms_norm_fp8(x, weight, eps, residual, pow2_scales)
    return _call(stream, _ops.rms_norm_fp8, x, weight, eps, residual, pow2_scales)


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, param_dtype=None, weight_grad: bool = True, stream=None):
    """Gradients (dx, dweight) of rms_norm: dx of x and of the residual alike, with dh, the gradient that h has
    from elsewhere, added.  dweight is of the weight's type (without a weight: ``param_dtype``, float32 or by
    default h's type), or None where it is not asked for."""
    if param_dtype is not None and param_dtype != torch.float32 and param_dtype != h.dtype:
        raise TypeError(f"param_dtype: {param_dtype} is neither {h.dtype} nor float32")
    args = dy, h, weight, rstd, dh, param_dtype == torch.float32, weight_grad
    if stream is None:
        return _ops.rms_norm_backward(*args)
    return _call(stream, _ops.rms_norm_backward, *args)


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


_SCORES = {"sigmoid": native.SCORE_SIGMOID, "softmax": native.SCORE_SOFTMAX}


def _score(name):
    if name not in _SCORES:
        raise ValueError(f"score: {name!r} is not one of {', '.join(map(repr, _SCORES))}")
    return _SCORES[name]


def route_scores(logits, topk: int, *, score: str = "sigmoid", bias=None, groups: int = 1, topk_groups: int | None = None,
                 group_top: int = 2, renormalize: bool = True, scale: float = 1.0, token_mask=None, stream=None):
    """Top-k experts of each token by the ``score`` ("sigmoid" or "softmax") of its logits [T, E], and their
    gate weights, FusedMoE.forward's (topk_idx int64, topk_w fp32) [T, topk].

    The choice goes by score + bias (fp32 [E]).  With ``groups`` of E/groups neighbouring experts, the
    ``topk_groups`` (default: all) groups with the largest sums of their ``group_top`` (1 or 2) best stay (a group
    with one expert that can be chosen is scored by that one).  The weights are the chosen scores without the
    bias, divided by their sum (``renormalize``), times ``scale``.  Values are compared as in 64 bits; ties, -inf
    logits and ``token_mask`` as in ``route_topk``."""
    args = (logits, topk, _score(score), bias, groups, groups if topk_groups is None else topk_groups, group_top, renormalize, scale,
            token_mask)
    if stream is None:
        return _ops.route_scores(*args)
    return _call(stream, _ops.route_scores, *args)


def route_scores_backward(dw, idx, w, logits, *, score: str = "sigmoid", renormalize: bool = True, scale: float = 1.0, stream=None):
    """Gradient of the logits (their type) from dw, that of route_scores' gate weights (fp32 [T, topk])."""
    args = dw, idx, w, logits, _score(score), renormalize, scale
    if stream is None:
        return _ops.route_scores_backward(*args)
    return _call(stream, _ops.route_scores_backward, *args)


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


# -------------------------------------------------------------- activation, 8-bit rows ----
def swiglu(gu, *, stream=None):
    """silu(gate) * up of rows of gate and up, gu [M, 2*I] (gate first; rows may be strided): [M, I]."""
    if stream is None:
        return _ops.swiglu(gu, False)
    return _call(stream, _ops.swiglu, gu, False)


def swiglu_backward(dact, gu, *, stream=None):
    """Gradient of swiglu's gu from dact [M, I]."""
    if stream is None:
        return _ops.swiglu_backward(dact, gu)
    return _call(stream, _ops.swiglu_backward, dact, gu)


def swiglu_checkpoint(gu, *, stream=None):
    """swiglu that keeps gu in 8 bits for its backward pass: (act, codes, scales).  32 neighbours of gate or
    of up share a scale byte b, and their codes n (int8 [M, 2*I]) stand for n * 2^(b - 133); scales uint8
    [M, 2*ceil(I/32)].  The largest of 32 keeps 6 to 7 bits; a NaN or an infinity makes its 32 NaN."""
    if stream is None:
        return _ops.swiglu(gu, True)
    return _call(stream, _ops.swiglu, gu, True)


def swiglu_checkpoint_backward(dact, codes, scales, *, stream=None):
    """(dgu, act) from dact [M, I] and what swiglu_checkpoint kept: the gradient of the values that the
    codes stand for, and their activation again, for the down weights' gradient."""
    if stream is None:
        return _ops.swiglu_checkpoint_backward(dact, codes, scales)
    return _call(stream, _ops.swiglu_checkpoint_backward, dact, codes, scales)


def checkpoint_rows(x, *, stream=None):
    """Rows [M, H] in swiglu_checkpoint's 8-bit format: (codes int8 [M, H], scales uint8 [M, ceil(H/32)])."""
    if stream is None:
        return _ops.checkpoint_rows(x)
    return _call(stream, _ops.checkpoint_rows, x)


_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}


def restore_rows(codes, scales, dtype, *, stream=None):
    """The rows that checkpoint_rows' codes and scales stand for, in ``dtype``."""
    if dtype not in _DTYPES:
        raise TypeError(f"dtype: {dtype} is not float32, bfloat16 or float16")
    if stream is None:
        return _ops.restore_rows(codes, scales, _DTYPES[dtype])
    return _call(stream, _ops.restore_rows, codes, scales, _DTYPES[dtype])


def get_error(stream=None) -> int:
    """Waits for ``stream`` (default: the current stream), then returns (and clears) the sticky status
    of the grouped products' bounded waits: 0 or MOE_ERR_TIMEOUT.  After the latter what they wrote is
    undefined.  The status is the device's: one that another thread asked for is cleared."""
    if stream is None:
        return _ops.get_error()
    return _call(stream, _ops.get_error)
