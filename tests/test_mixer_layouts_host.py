"""What a call keeps of its layout is found again by what it holds, never by the
identity of an option."""
import torch

from memory_bound_cnn_wtconv2d_gb300 import blockops, mixerops


def test_an_eps_that_changes(monkeypatch):
    monkeypatch.setattr(mixerops._c, "_on_cuda", lambda t: True)
    x, eps = torch.zeros(6, 64), torch.tensor(1e-6)
    first = mixerops._rms_layout(x, None, None, eps, ("x", "residual"))
    eps.fill_(0.5)
    second = mixerops._rms_layout(x, None, None, eps, ("x", "residual"))
    assert first.desc.eps != second.desc.eps == 0.5
    assert mixerops._rms_layout(x, None, None, 0.5, ("x", "residual")) is second


def test_an_eps_of_the_other_operators_that_changes(monkeypatch):
    class Layout:
        def __init__(self, x, dy, num_groups, eps, activation):
            self.eps = float(eps)

    class Lib:
        def wtconv_ns_workspace_size(self, ref):
            return 0

    monkeypatch.setattr(blockops, "_GnLayout", Layout)
    monkeypatch.setattr(blockops, "_LAYOUTS", {})
    monkeypatch.setattr(blockops, "_NS_DESCS", {})
    monkeypatch.setattr(blockops, "lib", Lib)
    x, eps = torch.zeros(2, 6, 64), torch.tensor(1e-5)
    stack = type("Stack", (), dict(m=8, n=8, dtype=torch.float32, device=torch.device("cpu")))
    first = blockops._gn_layout(x, None, 4, eps, "none"), blockops._ns_desc(stack, 1, 5, (1.0, 2.0, eps), eps)
    eps.fill_(0.25)
    second = blockops._gn_layout(x, None, 4, eps, "none"), blockops._ns_desc(stack, 1, 5, (1.0, 2.0, eps), eps)
    assert first[0].eps != second[0].eps == 0.25
    a, b = first[1][0]._obj, second[1][0]._obj
    assert a.eps != b.eps == 0.25 and a.c != b.c == 0.25
