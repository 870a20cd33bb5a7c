"""The block operators inside autograd: what is asked for, and what may not be
used any more."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


@pytest.mark.parametrize("shape,G", [((2, 6, 6, 24), 3), ((2, 90, 100, 48), 8)])
def test_only_the_gradients_asked_for(ops, shape, G):
    torch.manual_seed(0)
    x, dy = torch.randn(shape, device="cuda"), torch.randn(shape, device="cuda")
    w, b = torch.randn(shape[-1], device="cuda"), torch.randn(shape[-1], device="cuda")
    _, mean, rstd = ops.wtconv_gn_act_fwd(x, G, w, b, activation="silu")
    every = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, G, w, b, activation="silu")
    for need_w in (True, False):
        for need_b in (True, False):
            got = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, G, w, b, activation="silu", need_dweight=need_w, need_dbias=need_b)
            assert torch.equal(got[0], every[0])
            for k, need in ((1, need_w), (2, need_b)):
                assert (got[k] is not None) == need
                assert not need or torch.equal(got[k], every[k])


@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
def test_frozen_parameters_cost_no_sums(ops, monkeypatch, weight, bias):
    from memory_bound_cnn_wtconv2d_gb300.norm import GroupNormAct
    m = GroupNormAct(4, 16, activation="gelu", device="cuda")
    m.weight.requires_grad_(weight)
    m.bias.requires_grad_(bias)
    asked = []
    real = ops.wtconv_gn_act_bwd

    def spy(*args, **kw):
        asked.append((kw["need_dweight"], kw["need_dbias"]))
        return real(*args, **kw)

    monkeypatch.setattr(ops, "wtconv_gn_act_bwd", spy)
    x = torch.randn(2, 5, 6, 16, device="cuda", requires_grad=True)
    m(x).square().sum().backward()
    assert asked == [(weight, bias)]
    assert torch.isfinite(x.grad).all() and (m.weight.grad is not None, m.bias.grad is not None) == (weight, bias)
