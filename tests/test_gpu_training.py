"""The operators together: the trainable block's output and gradients against a plain 64-bit block,
the example's training run, and the trained weights through the fused FP8 layer.

Tolerances: the block rounds to bf16 (u = 2^-8) after the norm, each product, the SwiGLU and the
combine; a relative error of the sums of a few such roundings stays below 8u of the whole tensor's
norm, forward and (through twice as many steps) 16u backward.
"""
import os
import sys

import pytest
import torch

from combine_persistent_warp_gb300 import ops, training

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U16 = 2.0 ** -8


def _plain(block, x, idx, mask=None):
    """The block in 64 bits with the experts chosen as given; returns output and parameters' leaves."""
    p = {n: v.detach().double().requires_grad_() for n, v in block.named_parameters()}
    x = x.detach().double().requires_grad_()
    mean = x.mean(1, keepdim=True)
    h = (x - mean) * ((x - mean).square().mean(1, keepdim=True) + block.eps).rsqrt() * p["norm_weight"] + p["norm_bias"]
    logits = h @ p["router"].t()
    w = torch.softmax(logits.gather(1, idx.clamp_min(0)), 1)
    out = x
    for e in range(block.E):
        gu = h @ p["w_gate_up"][e].t()
        y = (torch.nn.functional.silu(gu[:, :block.I]) * gu[:, block.I:]) @ p["w_down"][e].t()
        out = out + ((idx == e) * w).sum(1, keepdim=True) * y
    return out, x, p


@pytest.mark.parametrize("T,E,H,I,topk,masked", [(1, 4, 64, 64, 2, False), (300, 8, 256, 128, 2, False), (257, 5, 136, 72, 3, True)])
def test_block_against_a_plain_one(T, E, H, I, topk, masked):
    torch.manual_seed(1)
    block = training.MoEBlock(E, H, I, topk, std=0.1).cuda()
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    mask = (torch.rand(T, device="cuda") < 0.7) if masked else None
    out = block(x, mask)
    seen = []
    keep = ops.expert_order
    ops.expert_order = lambda idx, E, **k: (seen.append(idx), keep(idx, E, **k))[1]
    try:
        assert torch.equal(block(x, mask), out)          # the same bits again
    finally:
        ops.expert_order = keep
    idx = seen[0]
    if masked:
        assert (idx[~mask] == -1).all() and torch.equal(out[~mask], x[~mask])
    ref, rx, rp = _plain(block, x, idx)
    d = torch.randn_like(out)
    out.backward(d)
    ref.backward(d.double())
    rel = lambda a, b: ((a.double() - b).norm() / b.norm().clamp_min(1e-30)).item()
    assert rel(out, ref) <= 8 * U16
    assert rel(x.grad, rx.grad) <= 16 * U16
    for n, v in block.named_parameters():
        assert rel(v.grad, rp[n].grad) <= 16 * U16, n
    assert ops.get_error() == 0


def test_example_trains_and_serves():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_moe_block as ex
    block, first, last = ex.train(steps=40, tokens=1024)
    assert last < 0.8 * first
    # FP8 (e4m3) operands carry 2^-4 relative steps: about 3% a tensor, three tensors deep
    assert ex.serve(block, tokens=256) < 0.15


def test_expanded_gradients():
    """The gradient of a plain sum is an expanded scalar: it reaches the kernels as real rows."""
    torch.manual_seed(2)
    block = training.MoEBlock(4, 64, 64, 2, std=0.1).cuda()
    x = torch.randn(20, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    block(x).sum().backward()
    g = x.grad.clone()
    x.grad = None
    block(x).backward(torch.ones(20, 64, device="cuda", dtype=torch.bfloat16))
    assert torch.equal(g, x.grad)
