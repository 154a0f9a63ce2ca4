"""Trains a small Mixture-of-Experts block on a synthetic target, then serves it through the fused
FP8 layer and compares the two.

    python examples/train_moe_block.py [--steps 60] [--tokens 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_persistent_warp_gb300 import ops  # noqa: E402
from combine_persistent_warp_gb300.training import MoEBlock  # noqa: E402


def train(steps: int = 60, tokens: int = 2048, E: int = 8, H: int = 256, I: int = 128, topk: int = 2, lr: float = 5e-3, seed: int = 0):
    """Fits block(x) to x + f(x) for a fixed f; returns (block, first loss, last loss)."""
    torch.manual_seed(seed)
    block = MoEBlock(E, H, I, topk, std=0.05).cuda()
    target = torch.randn(H, H, device="cuda") / H ** 0.5
    # fp32 master weights beside the 16-bit ones that the kernels read
    master = [p.detach().float().clone() for p in block.parameters()]
    opt = torch.optim.Adam(master, lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, H, device="cuda", dtype=torch.bfloat16)
        want = x.float() + torch.tanh(x.float() @ target)
        loss = (block(x).float() - want).square().mean()
        block.zero_grad(set_to_none=True)
        loss.backward()
        for m, p in zip(master, block.parameters()):
            m.grad = p.grad.float()
        opt.step()
        with torch.no_grad():
            for m, p in zip(master, block.parameters()):
                p.copy_(m)
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()
    if status := ops.get_error():
        raise RuntimeError(f"device status {status}")
    return block, losses[0], losses[-1]


def serve(block, tokens: int = 512):
    """Relative difference of the fused FP8 layer's output from the trained block's, on the MoE part."""
    x = torch.randn(tokens, block.H, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        full = block(x).float() - x.float()
    layer = block.serving_layer(tokens)
    fp8 = block.serve(layer, x).float() - x.float()
    torch.cuda.synchronize()
    status = layer.get_error() or ops.get_error()
    layer.close()
    if status:
        raise RuntimeError(f"device status {status}")
    return ((fp8 - full).norm() / full.norm()).item()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    block, first, last = train(a.steps, a.tokens)
    print(f"loss {first:.4f} -> {last:.4f} in {a.steps} steps of {a.tokens} tokens")
    print(f"fused FP8 layer: {serve(block):.3f} relative difference from the bf16 block")


if __name__ == "__main__":
    main()
