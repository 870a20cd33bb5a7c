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


def test_a_graph_that_saved_a_weight_is_not_used_after_the_step(ops):
    # as after any in-place operation: the gradient would be that of other weights
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    p = torch.nn.Parameter(torch.randn(24, 32, device="cuda"))
    x = torch.randn(5, 32, device="cuda", requires_grad=True)
    opt = Muon([p], lr=0.1)
    loss = torch.nn.functional.linear(x, p).square().sum()
    loss.backward(retain_graph=True)
    version = p._version
    opt.step()
    assert p._version > version
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_given_outputs_count_as_written(ops):
    x = torch.randn(2, 9, 16, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
    g, o = torch.randn(30, 40, device="cuda"), torch.empty(30, 40, device="cuda")
    given = [y, mean, rstd, dx, dw, db, o]
    before = [t._version for t in given]
    ops.wtconv_gn_act_fwd(x, 4, y=y, mean=mean, rstd=rstd)
    ops.wtconv_gn_act_bwd(x, x, mean, rstd, 4, dx=dx, dweight=dw, dbias=db)
    ops.wtconv_orthogonalize(g, out=o)
    assert all(t._version > v for t, v in zip(given, before))
    assert x._version == 0 and g._version == 0
    with torch.inference_mode():  # tensors without a version
        w = torch.randn(30, 40, device="cuda")
        ops.wtconv_muon_step(w, g, torch.zeros(30, 40, device="cuda"), lr=0.1)
