"""Residual blocks on the wavelet layer, and the optimisers of their parameters.

WTConv2d mixes space (NCHW planes); its output goes to channels last, through
a norm, pointwise matrices with an activation between them, and back onto the
input.
"""
from __future__ import annotations

import torch

from .layer import WTConv2d
from .mixer import GatedLinear, GatedLinear8, RMSNormAdd
from .muon import Muon
from .norm import GroupNormAct


class WTConvBlock(torch.nn.Module):
    """x + W2 gelu(norm(W1 norm(wtconv(x)))) on NCHW activations: the first norm
    without, the second with its activation.  The pointwise matrices are
    [hidden, C] and [C, hidden], hidden = expand * C."""

    def __init__(self, channels: int, kernel_size: int = 5, levels: int = 1, num_groups: int = 8, expand: int = 4,
                 device=None):
        super().__init__()
        hidden = expand * channels
        self.wtconv = WTConv2d(channels, kernel_size, levels, device=device)
        self.norm1 = GroupNormAct(num_groups, channels, device=device)
        self.up = torch.nn.Linear(channels, hidden, bias=False, device=device)
        self.norm2 = GroupNormAct(num_groups, hidden, activation="gelu", device=device)
        self.down = torch.nn.Linear(hidden, channels, bias=False, device=device)

    def forward(self, x):
        y = self.wtconv(x).permute(0, 2, 3, 1).contiguous()
        y = self.norm2(self.up(self.norm1(y)))
        return x + self.down(y).permute(0, 3, 1, 2)


class WTConvGatedBlock(torch.nn.Module):
    """t + W3 (act(W1 n) * (W2 n)) with t = x + wtconv(x) and n = rmsnorm(t), on NCHW
    activations: a gated channel mixer behind the layer.  W1 and W2 are [hidden, C],
    W3 is [C, hidden]; hidden is 8 / 3 C to a multiple of 16 unless given, which
    makes the three as large as the two of an expansion of four."""

    def __init__(self, channels: int, kernel_size: int = 5, levels: int = 1, hidden: int | None = None,
                 activation: str = "silu", device=None):
        super().__init__()
        hidden = max(16, round(channels / 6) * 16) if hidden is None else hidden
        self.wtconv = WTConv2d(channels, kernel_size, levels, device=device)
        self.norm = RMSNormAdd(channels, device=device)
        self.mix = GatedLinear(channels, hidden, activation, device=device)
        self.down = torch.nn.Linear(hidden, channels, bias=False, device=device)

    def quantize_(self):
        """From here on for inference alone: the norm's output and the gated matrices in
        8 bits (e4m3, a scale for each pixel and each hidden unit)."""
        if not isinstance(self.mix, GatedLinear8):
            self.mix = GatedLinear8(self.mix)
        return self

    def forward(self, x):
        a, r = self.wtconv(x).permute(0, 2, 3, 1).contiguous(), x.permute(0, 2, 3, 1).contiguous()
        if isinstance(self.mix, GatedLinear8):
            q, scale, total = self.norm.forward_8bit(a, r)
            h = self.mix(q, scale, self.down.weight.dtype)
        else:
            y, total = self.norm(a, r)
            h = self.mix(y)
        return (total + self.down(h)).permute(0, 3, 1, 2)


def block_optimizers(module: torch.nn.Module, lr: float = 0.02, other_lr: float = 1e-3, weight_decay: float = 0.0):
    """(Muon over the matrices of the module's linear layers, gated ones among them,
    AdamW over every other parameter).  weight_decay is that of both."""
    matrices = [m.weight for m in module.modules() if isinstance(m, torch.nn.Linear)]
    matrices += [w for m in module.modules() if isinstance(m, GatedLinear) for w in (m.gate, m.up)]
    taken = {id(p) for p in matrices}
    others = [p for p in module.parameters() if id(p) not in taken]
    return Muon(matrices, lr=lr, weight_decay=weight_decay), torch.optim.AdamW(others, lr=other_lr, weight_decay=weight_decay)
