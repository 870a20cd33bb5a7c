"""Clipping of a module's gradients by their global norm."""
from __future__ import annotations

import torch

from . import mixerops as _m


def clip_grad_norm_(parameters, max_norm: float, *, eps: float = 1e-6, error_if_nonfinite: bool = False):
    """Multiplies the gradients of `parameters` in place by min(1, max_norm / (norm +
    eps)), norm the root of the sum of squares of them all, which it returns
    (float32, on the gradients' device).  Parameters without a gradient count
    for nothing; one that comes twice counts once.  error_if_nonfinite reads the
    gradients once more and waits for the norm, and raises before anything is scaled.

    Narrower than torch.nn.utils.clip_grad_norm_: the norm is the 2-norm (its third
    argument is none here), and gradients are float32, float16 or bfloat16 on one GPU,
    dense, of elements that fill a stretch of memory each; two parameters with one
    gradient, or gradients that overlap, are refused (ValueError)."""
    params = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = list({id(p): p.grad for p in params if p.grad is not None}.values())
    if not grads:
        return torch.zeros(())
    if error_if_nonfinite:
        norm = _m.wtconv_grad_norm(grads)
        if not torch.isfinite(norm):
            raise RuntimeError(f"the global norm of the gradients is {float(norm)}")
    return _m.wtconv_clip_grads(grads, max_norm, eps=eps)
