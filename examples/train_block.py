"""Trains one MoE block on synthetic data with clipped gradients:

    python examples/train_block.py [--tokens 512 --steps 20]

The block learns to reproduce a fixed random map of its input; the printed loss
falls and the gradients' norm is what the clipping saw.  Float32 master weights
are updated by plain gradient descent and copied to the block's bf16 weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_sigmoid_amd as moe                                # noqa: E402
from fp8_block_scaled_sigmoid_amd.train import BlockWeights, MoEBlock   # noqa: E402


def make_block(H, I, N, k, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=gen)

    master = {"w_router": normal(N, H, std=0.05), "w1": normal(N + 1, 2 * I, H, std=H ** -0.5),
              "w2": normal(N + 1, H, I, std=I ** -0.5), "w_pre": torch.ones(H, device="cuda"),
              "w_post": torch.ones(H, device="cuda"), "gate": torch.full((H,), 0.5, device="cuda")}
    bf16 = {n: master[n].bfloat16() for n in ("w_router", "w1", "w2")}
    weights = BlockWeights(bias=torch.zeros(N, device="cuda"), **{**master, **bf16})
    return MoEBlock(weights, k), master


def train(tokens=512, steps=20, H=256, I=128, N=16, k=2, lr=2.0, max_norm=0.05, report=print):
    block, master = make_block(H, I, N, k)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(tokens, H, device="cuda").normal_(generator=gen)
    target = x + 0.3 * x @ torch.empty(H, H, device="cuda").normal_(0, H ** -0.5, generator=gen)
    losses = []
    for step in range(steps):
        r, _, saved = block.forward(x)
        diff = r - target
        losses.append(diff.square().mean())
        block.backward(saved, diff * (2.0 / diff.numel()))
        norm, coef = block.clip(max_norm)
        for name, m in master.items():
            m.sub_(block.grads[name], alpha=lr)
            if name in ("w_router", "w1", "w2"):
                getattr(block.w, name).copy_(m)
        moe.moe_bias_update(block.w.bias, saved[-1], tokens, k, 1e-3)
        report(f"step {step:3d}  loss {losses[-1].item():.4f}  gradient norm {norm.item():.4f}  "
               f"scaled by {coef.item():.3f}")
    return [v.item() for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    train(a.tokens, a.steps)
