"""The gated channel mixer as torch autograd functions / modules.

The activations are channels last: [..., C], each pixel one row of C values.
RMSNormAdd adds the residual and norms a pixel's channels, GatedLinear is the
pair of pointwise matrices with the activation and the product between them,
GatedLinear8 its 8-bit form for inference.
"""
from __future__ import annotations

import math

import torch

from . import blockops as _b
from . import mixerops as _m


class RMSNormAddFunction(torch.autograd.Function):
    """(y, total).  One backward, by the kernels; no second derivative, forward
    mode or vmap."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        y, total, rstd = _m.wtconv_rms_norm_fwd(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(total, rstd, weight)
        ctx.set_materialize_grads(False)
        return y, total

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dtotal):
        total, rstd, weight = ctx.saved_tensors
        need_x, need_r, need_w, _ = ctx.needs_input_grad
        if dy is None:  # only the sum was used
            return dtotal, dtotal, torch.zeros_like(weight) if need_w else None, None
        like = lambda t: None if t is None else t.contiguous().to(total.dtype)  # noqa: E731
        dx, dw = _m.wtconv_rms_norm_bwd(like(dy), total, rstd, weight, dtotal=like(dtotal), need_dweight=need_w)
        return dx if need_x else None, dx if need_r else None, dw, None


class RMSNormFunction(torch.autograd.Function):
    """The norm without a residual."""

    @staticmethod
    def forward(ctx, x, weight, eps):
        y, _, rstd = _m.wtconv_rms_norm_fwd(x, weight, eps=eps)
        ctx.save_for_backward(x, rstd, weight)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, rstd, weight = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = _m.wtconv_rms_norm_bwd(dy.contiguous().to(x.dtype), x, rstd, weight, need_dweight=need[1])
        return dx if need[0] else None, dw, None


def rms_norm_add(x, residual, weight=None, eps=1e-6):
    """(y, total): total = x + residual, y its root-mean-square norm times weight."""
    return RMSNormAddFunction.apply(x, residual, weight, eps)


def rms_norm(x, weight=None, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis."""
    return RMSNormFunction.apply(x, weight, eps)


class RMSNormAdd(torch.nn.Module):
    """Root-mean-square norm over channels-last activations [..., C], of x, or of
    x + residual, whose sum it returns beside its norm: norm(x) is y, norm(x,
    residual) is (y, total).  Parameter (float32): weight [C] (init 1), absent with
    affine=False."""

    def __init__(self, channels: int, eps: float = 1e-6, affine: bool = True, device=None):
        super().__init__()
        if not (isinstance(channels, int) and 1 <= channels <= 16384):
            raise ValueError(f"channels must be an int in [1, 16384], got {channels!r}")
        self.channels, self.eps = channels, eps
        self.weight = torch.nn.Parameter(torch.ones(channels, device=device, dtype=torch.float32)) if affine else None

    def extra_repr(self):
        return f"{self.channels}, eps={self.eps}, affine={self.weight is not None}"

    def _check(self, x):
        if x.shape[-1] != self.channels:
            raise ValueError(f"expected channels-last activations of {self.channels} channels, got {tuple(x.shape)}")

    def forward(self, x, residual=None):
        self._check(x)
        if residual is None:
            return rms_norm(x, self.weight, self.eps)
        return rms_norm_add(x, residual, self.weight, self.eps)

    def forward_8bit(self, x, residual=None):
        """(q, scale, total): the norm in 8 bits, for GatedLinear8; no gradient."""
        self._check(x)
        _no_gradient()
        return _m.wtconv_rms_norm_q8(x, self.weight, residual=residual, eps=self.eps)


def _no_gradient():
    if torch.is_grad_enabled():
        raise RuntimeError("8-bit inference has no gradient: call it under torch.no_grad()")


class GatedFunction(torch.autograd.Function):
    """Keeps x and the matrices; the backward makes their products again.  One
    backward, by the kernels; no second derivative, forward mode or vmap."""

    @staticmethod
    def forward(ctx, x, gate, up, activation):
        ctx.save_for_backward(x, gate, up)
        ctx.activation = activation
        return _m.wtconv_gated_fwd(x, gate, up, activation=activation)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, gate, up = ctx.saved_tensors
        need_x, need_gate, need_up, _ = ctx.needs_input_grad
        # an upstream gradient may come broadcast (stride 0) or in another order of axes
        dx, dgate, dup = _m.wtconv_gated_bwd(dh.contiguous().to(x.dtype), x, gate, up, activation=ctx.activation,
                                             need_dx=need_x, need_dweights=need_gate or need_up)
        return dx, dgate if need_gate else None, dup if need_up else None, None


def gated_linear(x, gate, up, activation="silu"):
    """act(x gate^T) * (x up^T); under autocast in its type."""
    if torch.is_autocast_enabled("cuda"):
        dtype = torch.get_autocast_dtype("cuda")
        x, gate, up = x.to(dtype), gate.to(dtype), up.to(dtype)
    return GatedFunction.apply(x, gate, up, activation)


class GatedLinear(torch.nn.Module):
    """act(x gate^T) * (x up^T) on rows [..., C]: two matrices [hidden, C] without
    biases, an activation ("none", "silu" or "gelu") and the product of the two."""

    def __init__(self, channels: int, hidden: int, activation: str = "silu", device=None, dtype=None):
        super().__init__()
        if not all(isinstance(v, int) and 1 <= v <= 65536 for v in (channels, hidden)):
            raise ValueError(f"channels and hidden must be ints in [1, 65536], got {channels!r} and {hidden!r}")
        if activation not in _b.ACT_CODES:
            raise ValueError(f"activation must be one of none, silu, gelu, got {activation!r}")
        self.channels, self.hidden, self.activation = channels, hidden, activation
        bound = 1.0 / math.sqrt(channels)
        make = lambda: torch.nn.Parameter(torch.empty(hidden, channels, device=device, dtype=dtype).uniform_(-bound, bound))  # noqa: E731
        self.gate, self.up = make(), make()

    def extra_repr(self):
        return f"{self.channels}, {self.hidden}, activation={self.activation}"

    def forward(self, x):
        if x.shape[-1] != self.channels:
            raise ValueError(f"expected channels-last activations of {self.channels} channels, got {tuple(x.shape)}")
        return gated_linear(x, self.gate, self.up, self.activation)


class GatedLinear8(torch.nn.Module):
    """GatedLinear for inference, in 8 bits: its matrices as e4m3 with a scale for each
    hidden unit, on activations that ``RMSNormAdd.forward_8bit`` hands over."""

    def __init__(self, linear: GatedLinear):
        super().__init__()
        if linear.channels % 16:
            raise ValueError(f"8-bit operands: the {linear.channels} channels must be a multiple of 16")
        self.channels, self.hidden, self.activation = linear.channels, linear.hidden, linear.activation
        for name in ("gate", "up"):
            q, scale = _m.wtconv_quantize_rows(getattr(linear, name).detach())
            self.register_buffer(name, q)
            self.register_buffer(name + "_scale", scale)

    def extra_repr(self):
        return f"{self.channels}, {self.hidden}, activation={self.activation}, 8 bits"

    def forward(self, q, scale, dtype):
        _no_gradient()
        return _m.wtconv_gated_q8(q, scale, self.gate, self.gate_scale, self.up, self.up_scale, activation=self.activation,
                                  dtype=dtype)
