"""Group norm with an activation as a torch autograd function / module.

The activations are channels last: [N, ..., C], each pixel one row of C
values, as the pointwise matrices of a block read them.
"""
from __future__ import annotations

import torch

from . import blockops as _b


class GroupNormActFunction(torch.autograd.Function):
    """One backward, by the kernels.  No second derivative, no forward mode, no
    vmap or torch.func: torch raises where one is asked for."""

    @staticmethod
    def forward(ctx, x, weight, bias, num_groups, eps, activation):
        y, mean, rstd = _b.wtconv_gn_act_fwd(x, num_groups, weight, bias, eps=eps, activation=activation)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.num_groups, ctx.activation = num_groups, activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        # an upstream gradient may come broadcast (stride 0) or in another order of axes
        need = ctx.needs_input_grad
        dx, dw, db = _b.wtconv_gn_act_bwd(dy.contiguous().to(x.dtype), x, mean, rstd, ctx.num_groups, weight, bias,
                                          activation=ctx.activation, need_dweight=need[1], need_dbias=need[2])
        return (dx if need[0] else None, dw, db, None, None, None)


def group_norm_act(x, num_groups, weight=None, bias=None, eps=1e-5, activation="none"):
    """act(group_norm(x) * weight + bias) on channels-last x [N, ..., C]."""
    return GroupNormActFunction.apply(x, weight, bias, num_groups, eps, activation)


class GroupNormAct(torch.nn.Module):
    """Group norm over channels-last activations [N, ..., C], then an activation
    ("none", "silu" or "gelu").  Parameters (float32): weight [C] (init 1) and
    bias [C] (init 0), absent with affine=False."""

    def __init__(self, num_groups: int, channels: int, eps: float = 1e-5, activation: str = "none",
                 affine: bool = True, device=None):
        super().__init__()
        if not (isinstance(num_groups, int) and num_groups >= 1 and channels >= 1 and channels % num_groups == 0):
            raise ValueError(f"num_groups = {num_groups} must be a positive divisor of the {channels} channels")
        if activation not in _b.ACT_CODES:
            raise ValueError(f"activation must be one of none, silu, gelu, got {activation!r}")
        self.num_groups, self.channels, self.eps, self.activation = num_groups, channels, eps, activation
        f = dict(device=device, dtype=torch.float32)
        self.weight = torch.nn.Parameter(torch.ones(channels, **f)) if affine else None
        self.bias = torch.nn.Parameter(torch.zeros(channels, **f)) if affine else None

    def extra_repr(self):
        return (f"{self.num_groups}, {self.channels}, eps={self.eps}, activation={self.activation}, "
                f"affine={self.weight is not None}")

    def forward(self, x):
        if x.shape[-1] != self.channels:
            raise ValueError(f"expected channels-last activations of {self.channels} channels, got {tuple(x.shape)}")
        return group_norm_act(x, self.num_groups, self.weight, self.bias, self.eps, self.activation)
