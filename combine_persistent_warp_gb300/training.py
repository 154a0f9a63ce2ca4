"""Autograd functions over ``ops`` and a trainable Mixture-of-Experts block.

    block = MoEBlock(E, H, I, topk).cuda()
    y = block(x)                       # x + MoE(LayerNorm(x)), bf16 [T, H]
    y.float().square().mean().backward()

Every product, norm, router and row movement of the block, forward and backward, is one of the
framework's kernels; what is left to PyTorch is elementwise (SwiGLU, the residual sum) and the
small dense product with the router's weight.  With an RMS norm the residual that it adds is a
kernel's too, and with 8-bit checkpoints the SwiGLU:

    block = MoEBlock(E, H, I, topk, norm="rms", score="sigmoid", groups=8, topk_groups=4, balance=True, checkpoint=True)
    y = block(x, residual=stream)      # s + MoE(RMSNorm(s)), s = x + stream
    block.update_balance()             # between steps: the biases against the experts' loads

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


class _RMSNorm(Function):
    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        y, rstd, h = ops.rms_norm(x, weight, eps, residual=residual)
        ctx.save_for_backward(h, weight, rstd)
        ctx.set_materialize_grads(False)
        return y, h if residual is not None else None   # (without one h is x, no output of its own)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight, rstd = ctx.saved_tensors
        if dy is None:   # only the sum was used
            return dh, None, None, dh
        dx, dweight = ops.rms_norm_backward(_rows(dy), h, weight, rstd, dh=None if dh is None else _rows(dh),
                                            weight_grad=ctx.needs_input_grad[1])
        return dx, dweight, None, dx if ctx.needs_input_grad[3] else None


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


class _RouteScores(Function):
    @staticmethod
    def forward(ctx, logits, topk, options, token_mask):
        idx, w = ops.route_scores(logits, topk, token_mask=token_mask, **options)
        ctx.save_for_backward(idx, w, logits)
        ctx.options = {k: options[k] for k in ("score", "renormalize", "scale") if k in options}
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        idx, w, logits = ctx.saved_tensors
        return ops.route_scores_backward(dw.contiguous(), idx, w, logits, **ctx.options), None, None, None


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


class _SwiGLU(Function):
    @staticmethod
    def forward(ctx, gu, checkpoint):
        if checkpoint:
            act, *kept = ops.swiglu_checkpoint(gu)
        else:
            act, kept = ops.swiglu(gu), [gu]
        ctx.save_for_backward(*kept)
        return act

    @staticmethod
    @once_differentiable
    def backward(ctx, dact):
        kept = ctx.saved_tensors
        if len(kept) == 1:
            return ops.swiglu_backward(_rows(dact), *kept), None
        return ops.swiglu_checkpoint_backward(_rows(dact), *kept)[0], None


class _Experts(Function):
    """From the tokens' rows to the experts' weighted sums, with 8-bit checkpoints: between forward and backward
    it holds h, gate and up in 8 bits and, for the gate weights' gradient, the down products' rows in 8 bits; the
    gathered rows and the activation are made again."""

    @staticmethod
    def forward(ctx, h, rows, offsets, w, w_gate_up, w_down):
        gu = ops.grouped_mm(ops.gather_rows(h, rows, offsets), w_gate_up, offsets)
        act, *kept = ops.swiglu_checkpoint(gu)
        y = ops.grouped_mm(act, w_down, offsets)
        ctx.save_for_backward(h, rows, offsets, w, w_gate_up, w_down, *kept, *(ops.checkpoint_rows(y) if ctx.needs_input_grad[3] else ()))
        return ops.combine_rows(y, rows, w)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        h, rows, offsets, w, w_gate_up, w_down, codes, scales, *kept = ctx.saved_tensors
        dout = _rows(dout)
        want_h, _, _, want_w, want_gate_up, want_down = ctx.needs_input_grad
        # (without the gate weights' gradient the rows themselves are not read: their shape alone counts)
        y = ops.restore_rows(*kept, dout.dtype) if want_w else dout.new_empty(rows.numel(), dout.shape[1])
        dy, dw = ops.combine_rows_backward(dout, y, rows, w, offsets, gate_grad=want_w)
        del y
        if not (want_h or want_gate_up or want_down):
            return None, None, None, dw, None, None
        dgu, act = ops.swiglu_checkpoint_backward(ops.grouped_mm_dx(dy, w_down, offsets), codes, scales)
        dw_down = ops.grouped_mm_dw(dy, act, offsets) if want_down else None
        del dy, act
        dw_gate_up = ops.grouped_mm_dw(dgu, ops.gather_rows(h, rows, offsets), offsets) if want_gate_up else None
        dh = ops.combine_rows(ops.grouped_mm_dx(dgu, w_gate_up, offsets), rows) if want_h else None
        return dh, None, None, dw, dw_gate_up, dw_down


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


def rms_norm(x, weight, eps: float = 1e-6, residual=None):
    """(y, h): the norm of h = x + residual (without a residual, of h = x)."""
    y, h = _RMSNorm.apply(x, weight, eps, residual)
    return y, x if h is None else h


def route_scores(logits, topk: int, token_mask=None, **options):
    """(topk_idx, topk_w): differentiable through topk_w.  ``options`` are ops.route_scores'."""
    return _RouteScores.apply(logits, topk, options, token_mask)


def swiglu(gu, checkpoint: bool = False):
    """silu(gate) * up; with ``checkpoint`` gu is kept for the backward pass in 8 bits."""
    return _SwiGLU.apply(gu, checkpoint and torch.is_grad_enabled())


def experts(h, order: ops.ExpertOrder, w, w_gate_up, w_down):
    """combine_rows(SwiGLU experts(gather_rows(h))) with 8-bit checkpoints: w_gate_up [E, 2I, H], w_down [E, H, I]."""
    if not torch.is_grad_enabled():   # the same bits, and nothing kept
        gu = ops.grouped_mm(ops.gather_rows(h, order.rows, order.offsets), w_gate_up, order.offsets)
        return ops.combine_rows(ops.grouped_mm(ops.swiglu(gu), w_down, order.offsets), order.rows, w)
    return _Experts.apply(h, order.rows, order.offsets, w, w_gate_up, w_down)


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
    :meth:`serve` runs a batch through it with the norm written straight into its FP8 rows.

    ``norm="rms"``: an RMS norm, and :meth:`forward` takes a ``residual`` that it adds on the way.
    ``score``: the router of ops.route_scores with ``groups``, ``topk_groups``, ``group_top``, ``renormalize`` and
    ``scale``; with ``balance`` it has a bias for each expert, which :meth:`update_balance` moves against the
    loads of the batches since.  ``checkpoint``: the experts' activations are kept in 8 bits (``experts``),
    and the SwiGLU is rounded once (without, PyTorch's rounds silu(gate) too, so that the last bits differ)."""

    def __init__(self, E: int, H: int, I: int, topk: int, *, eps: float = 1e-5, dtype=torch.bfloat16, std: float = 0.02,
                 norm: str = "layer", score: str | None = None, groups: int = 1, topk_groups: int | None = None, group_top: int = 2,
                 renormalize: bool = True, scale: float = 1.0, balance: bool = False, checkpoint: bool = False):
        super().__init__()
        if norm not in ("layer", "rms"):
            raise ValueError(f"norm: {norm!r} is not 'layer' or 'rms'")
        if score is None and (groups != 1 or topk_groups is not None or group_top != 2 or not renormalize or scale != 1.0 or balance):
            raise ValueError("groups, topk_groups, group_top, renormalize, scale and balance need a score")
        self.E, self.H, self.I, self.topk, self.eps = E, H, I, topk, eps
        self.norm, self.checkpoint = norm, checkpoint
        self.routing = None if score is None else dict(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top,
                                                       renormalize=renormalize, scale=scale)
        p = lambda *shape: nn.Parameter(torch.randn(*shape, dtype=torch.float32).mul_(std).to(dtype))
        self.norm_weight = nn.Parameter(torch.ones(H, dtype=dtype))
        if norm == "layer":
            self.norm_bias = nn.Parameter(torch.zeros(H, dtype=dtype))
        self.router = p(E, H)
        self.w_gate_up = p(E, 2 * I, H)
        self.w_down = p(E, H, I)
        self.register_buffer("balance_bias", torch.zeros(E, dtype=torch.float32) if balance else None)
        self.register_buffer("load", torch.zeros(E, dtype=torch.int64) if balance else None, persistent=False)

    def _apply(self, fn, recurse=True):
        # the biases move by less than a step of 16-bit numbers: a change of the block's type leaves them in fp32
        exact = self.balance_bias
        super()._apply(fn, recurse)
        if exact is not None and self.balance_bias.dtype != exact.dtype:
            self.balance_bias = exact.to(self.balance_bias.device)
        return self

    def _route(self, h, token_mask, choose, choose_scores):
        logits = h @ self.router.t()
        if self.routing is None:
            return choose(logits, self.topk, token_mask=token_mask)
        return choose_scores(logits, self.topk, token_mask=token_mask, bias=self.balance_bias, **self.routing)

    def forward(self, x, token_mask=None, *, residual=None):
        if residual is not None and self.norm != "rms":
            raise ValueError("a residual needs norm='rms'")
        # (an unrouted token's gradients are zeros, but zero times what padding may hold is not always zero)
        clean = lambda t: t if token_mask is None else t.masked_fill(~token_mask[:, None], 0)
        if self.norm == "layer":
            h = layer_norm(clean(x), self.norm_weight, self.norm_bias, self.eps)
        elif residual is None:
            h, _ = rms_norm(clean(x), self.norm_weight, self.eps)
        else:
            h, total = rms_norm(clean(x), self.norm_weight, self.eps, clean(residual))
            x = total if token_mask is None else torch.where(token_mask[:, None], total, x + residual)
        idx, w = self._route(h, token_mask, route_topk, route_scores)
        order = ops.expert_order(idx, self.E)
        if self.load is not None and self.training:
            self.load += order.offsets.diff()
        if self.checkpoint:
            return x + experts(h, order, w, self.w_gate_up, self.w_down)
        gate, up = grouped_mm(gather_rows(h, order), self.w_gate_up, order.offsets).chunk(2, dim=1)
        y = grouped_mm(torch.nn.functional.silu(gate) * up, self.w_down, order.offsets)
        return x + combine_rows(y, order, w)

    @torch.no_grad()
    def update_balance(self, rate: float = 1e-3):
        """Moves each expert's bias by ``rate`` towards the mean load of the training batches since the last
        call, and starts counting again."""
        if self.balance_bias is None:
            raise ValueError("the block has no balance")
        load = self.load.double()
        self.balance_bias += rate * torch.sign(load.mean() - load).float()
        self.load.zero_()

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
    def serve(self, layer, x, token_mask=None, *, residual=None):
        """x + FusedMoE(LayerNorm(x)), or with the block's RMS norm, router and residual: the norm's FP8 rows and the
        router's choice go to the fused layer."""
        if residual is not None and self.norm != "rms":
            raise ValueError("a residual needs norm='rms'")
        if self.norm == "layer":
            h = ops.layer_norm(x, self.norm_weight, self.norm_bias, self.eps)[0]
            q, sf = ops.layer_norm_fp8(x, self.norm_weight, self.norm_bias, self.eps)
        else:
            h, _, x = ops.rms_norm(x, self.norm_weight, self.eps, residual=residual)
            q, sf, _ = ops.rms_norm_fp8(x, self.norm_weight, self.eps)
        idx, w = self._route(h, token_mask, ops.route_topk, ops.route_scores)
        return x + layer.forward(q, sf, idx, w).to(x.dtype)
