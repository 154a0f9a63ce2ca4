"""Autograd functions over ``ops`` and a trainable Mixture-of-Experts block.

    block = MoEBlock(E, H, I, topk).cuda()
    y = block(x)                       # x + MoE(LayerNorm(x)), bf16 [T, H]
    y.float().square().mean().backward()

Every product, norm, router and row movement of the block, forward and backward, is one of the
framework's kernels; what is left to PyTorch is elementwise (SwiGLU, the residual sum) and the
small dense product with the router's weight.

The functions are differentiable once, and cannot be traced, compiled or mapped (``torch.func.vmap``).
The waits inside the grouped products are bounded; one that ran out shows in ``ops.get_error()``,
which a training program asks where it waits for the GPU anyway.
"""
from __future__ import annotations

import torch
from torch import nn
from torch.autograd import Function
from torch.autograd.function import once_differentiable

from . import ops


class _LayerNorm(Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ops.layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        _, weight_grad, bias_grad, _ = ctx.needs_input_grad   # (False for None, which may have no gradient)
        return *ops.layer_norm_backward(_rows(dy), x, weight, mean, rstd, param_dtype=ctx.bias_dtype, weight_grad=weight_grad,
                                        bias_grad=bias_grad), None


class _RouteTopk(Function):
    @staticmethod
    def forward(ctx, logits, topk, token_mask, renormalize):
        idx, w = ops.route_topk(logits, topk, token_mask=token_mask, renormalize=renormalize)
        ctx.save_for_backward(idx, w, logits)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        idx, w, logits = ctx.saved_tensors
        return ops.route_topk_backward(dw.contiguous(), idx, w, logits, renormalize=ctx.renormalize), None, None, None


class _GatherRows(Function):
    @staticmethod
    def forward(ctx, x, rows, offsets):
        ctx.save_for_backward(rows)
        return ops.gather_rows(x, rows, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        rows, = ctx.saved_tensors
        return ops.combine_rows(dout.contiguous(), rows), None, None


class _CombineRows(Function):
    @staticmethod
    def forward(ctx, y, rows, w, offsets):
        ctx.save_for_backward(y, rows, w, offsets)
        return ops.combine_rows(y, rows, w)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        y, rows, w, offsets = ctx.saved_tensors
        dy, dw = ops.combine_rows_backward(_rows(dout), y, rows, w, offsets, gate_grad=ctx.needs_input_grad[2])
        return dy, None, dw, None


class _GroupedMM(Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return ops.grouped_mm(x, w, offsets)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = _rows(dy)
        dx = ops.grouped_mm_dx(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = ops.grouped_mm_dw(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def _rows(t):
    """A gradient as the operators take matrices: rows that are contiguous, apart from each other and,
    where their width allows it, on 16-byte boundaries (autograd hands over expanded or transposed
    ones, of a sum for instance, and pieces of others that start anywhere)."""
    size = t.element_size()
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1] and (t.stride(0) * size) % 16 == 0 and t.data_ptr() % 16 == 0:
        return t
    if t.is_contiguous() and (t.shape[1] * size) % 16 != 0:
        return t
    # (contiguous() gives a contiguous tensor back as it is, wherever it starts)
    return t.clone(memory_format=torch.contiguous_format)


def layer_norm(x, weight, bias, eps: float = 1e-5):
    return _LayerNorm.apply(x, weight, bias, eps)


def route_topk(logits, topk: int, token_mask=None, renormalize: bool = True):
    """(topk_idx, topk_w): differentiable through topk_w."""
    return _RouteTopk.apply(logits, topk, token_mask, renormalize)


def gather_rows(x, order: ops.ExpertOrder):
    return _GatherRows.apply(x, order.rows, order.offsets)


def combine_rows(y, order: ops.ExpertOrder, w):
    return _CombineRows.apply(y, order.rows, w, order.offsets)


def grouped_mm(x, w, offsets):
    return _GroupedMM.apply(x, w, offsets)


class MoEBlock(nn.Module):
    """x + MoE(LayerNorm(x)) with SwiGLU experts, for training in bfloat16 or float16.

    The expert weights have the fused layer's shapes: ``w_gate_up`` [E, 2I, H] (rows 0..I-1 gate,
    I..2I-1 up) and ``w_down`` [E, H, I]; :meth:`serving_layer` quantises them into a FusedMoE, and
    :meth:`serve` runs a batch through it with the norm written straight into its FP8 rows."""

    def __init__(self, E: int, H: int, I: int, topk: int, *, eps: float = 1e-5, dtype=torch.bfloat16, std: float = 0.02):
        super().__init__()
        self.E, self.H, self.I, self.topk, self.eps = E, H, I, topk, eps
        p = lambda *shape: nn.Parameter(torch.randn(*shape, dtype=torch.float32).mul_(std).to(dtype))
        self.norm_weight = nn.Parameter(torch.ones(H, dtype=dtype))
        self.norm_bias = nn.Parameter(torch.zeros(H, dtype=dtype))
        self.router = p(E, H)
        self.w_gate_up = p(E, 2 * I, H)
        self.w_down = p(E, H, I)

    def forward(self, x, token_mask=None):
        # (an unrouted token's gradients are zeros, but zero times what padding may hold is not always zero)
        seen = x if token_mask is None else x.masked_fill(~token_mask[:, None], 0)
        h = layer_norm(seen, self.norm_weight, self.norm_bias, self.eps)
        idx, w = route_topk(h @ self.router.t(), self.topk, token_mask)
        order = ops.expert_order(idx, self.E)
        gate, up = grouped_mm(gather_rows(h, order), self.w_gate_up, order.offsets).chunk(2, dim=1)
        y = grouped_mm(torch.nn.functional.silu(gate) * up, self.w_down, order.offsets)
        return x + combine_rows(y, order, w)

    # ------------------------------------------------------------------- serving -------
    @torch.no_grad()
    def serving_layer(self, max_tokens: int):
        """A FusedMoE with these expert weights as FP8 (128x128 block scales)."""
        from .native import FusedMoE
        from .workloads import quantize_128x128

        gu = [quantize_128x128(w.float()) for w in self.w_gate_up]
        down = [quantize_128x128(w.float()) for w in self.w_down]
        cat = lambda parts, i: torch.stack([q[i] for q in parts])
        layer = FusedMoE(self.E, self.H, self.I, self.topk, 1).reserve(max_tokens)
        return layer.load_weights(cat(gu, 0), cat(gu, 1), cat(down, 0), cat(down, 1))

    @torch.no_grad()
    def serve(self, layer, x, token_mask=None):
        """x + FusedMoE(LayerNorm(x)): the norm's FP8 rows and the router's choice go to the fused layer."""
        h = ops.layer_norm(x, self.norm_weight, self.norm_bias, self.eps)[0]
        q, sf = ops.layer_norm_fp8(x, self.norm_weight, self.norm_bias, self.eps)
        idx, w = ops.route_topk(h @ self.router.t(), self.topk, token_mask=token_mask)
        return x + layer.forward(q, sf, idx, w).to(x.dtype)
