"""An optimiser for the matrices of a block: momentum, then an orthogonalised
direction (Newton-Schulz), then a decayed weight update, in one call per shape.
"""
from __future__ import annotations

import math

import torch

from . import blockops as _b


def shape_scale(m: int, n: int, rule: str = "spectral") -> float:
    """Factor on the learning rate of an m x n matrix: "spectral" keeps the size
    of the change that the matrix makes to its output, max(1, m / n) ** 0.5;
    "rms" gives every update the root mean square 0.2, 0.2 * max(m, n) ** 0.5."""
    if rule == "spectral":
        return math.sqrt(max(1.0, m / n))
    if rule == "rms":
        return 0.2 * math.sqrt(max(m, n))
    raise ValueError(f"scale rule must be spectral or rms, got {rule!r}")


class _FaultWatch:
    """The count of in-kernel waits that gave up on one device, copied behind every
    step and looked at before the next one, without a wait for the GPU."""

    def __init__(self, device):
        self.device = device
        self.count = torch.zeros(1, dtype=torch.int32, pin_memory=True)
        self.copy()
        torch.cuda.current_stream(device).synchronize()  # once: what others left in the count
        self.seen = int(self.count)

    def copy(self):
        _b.wtconv_block_device_faults_async(self.count, self.device)

    def check(self):
        now, before = int(self.count), self.seen
        self.seen = now
        if now > before:  # it only falls when someone reads and resets it
            raise RuntimeError(f"a wait inside the matrix kernels on {self.device} gave up since the last step: weights of "
                               "an earlier step, of this optimiser or of another, were left as they were")


class Muon(torch.optim.Optimizer):
    """Momentum with orthogonalised updates, for parameters that are matrices.

    A parameter of more than two axes (a pointwise convolution's [O, I, 1, 1])
    is taken as a matrix of its first axis by all the others.  Parameters of
    one shape and type take their step in one call.  Other parameters (norms,
    biases, depthwise kernels) belong to another optimiser.

    The kernels' waits are bounded; where one gave up, weights were left as they
    were, and a later ``step`` raises RuntimeError (the first one that starts
    after the GPU got there).
    """

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, steps: int = 5, coefficients=_b.NS_COEFFICIENTS, eps: float = 1e-7,
                 scale: str = "spectral"):
        if not (lr >= 0 and 0 <= momentum < 1 and weight_decay >= 0):
            raise ValueError("lr and weight_decay must not be negative, momentum must be in [0, 1)")
        shape_scale(1, 1, scale)
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay,
                                      steps=steps, coefficients=tuple(coefficients), eps=eps, scale=scale))
        for group in self.param_groups:
            for p in group["params"]:
                if p.dim() < 2:
                    raise ValueError(f"Muon takes matrices, got a parameter of shape {tuple(p.shape)}")
                if not p.is_contiguous():
                    raise ValueError("Muon takes contiguous parameters")

    def load_state_dict(self, state_dict):
        """As every optimiser's, but the buffers stay float32: the base class casts
        the state of 16-bit parameters to their type."""
        super().load_state_dict(state_dict)
        saved = [i for group in state_dict["param_groups"] for i in group["params"]]
        params = [p for group in self.param_groups for p in group["params"]]
        for i, p in zip(saved, params):
            entry = state_dict["state"].get(i)
            if entry and "buffer" in entry:
                self.state[p]["buffer"] = entry["buffer"].detach().to(p.device, torch.float32, copy=True).contiguous()

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        watches = self.__dict__.setdefault("_watches", {})
        for watch in watches.values():
            watch.check()
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        devices = set()
        for group in self.param_groups:
            stacks = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if not state:
                    state["buffer"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
                rows = p.shape[0]
                w, b = p.view(rows, -1), state["buffer"].view(rows, -1)
                g = p.grad.reshape(rows, -1)
                g = (g if g.is_contiguous() else g.contiguous()).to(p.dtype)
                stacks.setdefault((tuple(w.shape), p.dtype, p.device), []).append((w, g, b))
                devices.add(p.device)
            for (shape, _, device), entries in stacks.items():
                if device not in watches and device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
                    watches[device] = _FaultWatch(device)
                w, g, b = zip(*entries)
                _b.wtconv_muon_step(w, g, b, lr=group["lr"], momentum=group["momentum"], nesterov=group["nesterov"],
                                    weight_decay=group["weight_decay"], scale=shape_scale(*shape, group["scale"]),
                                    steps=group["steps"], coefficients=group["coefficients"], eps=group["eps"])
        for device in devices & watches.keys():
            watches[device].copy()
        return loss
