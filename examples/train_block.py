"""Trains a small classifier of two wavelet blocks on synthetic textures.

Each class is a sinusoidal grating of its own orientation and frequency under
noise; the blocks run WTConv2d, the group norms and the Muon optimiser of this
package together; with --gated the RMS norms and gated products, and the
gradients are clipped by their global norm.  Prints the loss as it goes, and the
final accuracy.

    python examples/train_block.py [--steps 60] [--channels 32] [--size 32] [--gated]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from memory_bound_cnn_wtconv2d_gb300.block import WTConvBlock, WTConvGatedBlock, block_optimizers  # noqa: E402
from memory_bound_cnn_wtconv2d_gb300.clip import clip_grad_norm_  # noqa: E402


def textures(batch, size, classes, generator, device):
    label = torch.randint(classes, (batch,), generator=generator, device=device)
    angle = label * (math.pi / classes)
    freq = 0.35 + 0.5 * (label % 2)
    phase = 2 * math.pi * torch.rand(batch, generator=generator, device=device)
    i = torch.arange(size, device=device, dtype=torch.float32)
    u = i[None, :, None] * angle.sin()[:, None, None] + i[None, None, :] * angle.cos()[:, None, None]
    image = torch.sin(u * freq[:, None, None] + phase[:, None, None])
    return image[:, None] + 0.5 * torch.randn(batch, 1, size, size, generator=generator, device=device), label


def train(steps=60, channels=32, size=32, batch=64, classes=6, device="cuda", seed=0, log=print, gated=False):
    torch.manual_seed(seed)
    generator = torch.Generator(device=device)
    generator.manual_seed(seed)
    stem = torch.nn.Conv2d(1, channels, 3, padding=1, device=device)
    make = ((lambda: WTConvGatedBlock(channels, levels=2, device=device)) if gated else
            (lambda: WTConvBlock(channels, levels=2, num_groups=4, device=device)))
    blocks = torch.nn.Sequential(*[make() for _ in range(2)])
    head = torch.nn.Linear(channels, classes, device=device)
    muon, adam = block_optimizers(blocks)
    rest = torch.optim.AdamW([*stem.parameters(), *head.parameters()], lr=3e-3)
    losses, accuracy = [], 0.0
    for step in range(steps):
        x, label = textures(batch, size, classes, generator, device)
        logits = head(blocks(stem(x)).mean(dim=(2, 3)))
        loss = torch.nn.functional.cross_entropy(logits, label)
        for o in (muon, adam, rest):
            o.zero_grad(set_to_none=True)
        loss.backward()
        if gated:
            clip_grad_norm_([*stem.parameters(), *blocks.parameters(), *head.parameters()], 1.0)
        for o in (muon, adam, rest):
            o.step()
        losses.append(float(loss.detach()))
        accuracy = float((logits.argmax(1) == label).float().mean())
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {losses[-1]:.4f}  accuracy {accuracy:.2f}")
    return losses, accuracy


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--channels", type=int, default=32)
    ap.add_argument("--size", type=int, default=32)
    ap.add_argument("--gated", action="store_true", help="blocks with a gated channel mixer, gradients clipped")
    a = ap.parse_args()
    train(a.steps, a.channels, a.size, gated=a.gated)
