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


def test_what_the_function_does_not_have_raises(ops):
    from memory_bound_cnn_wtconv2d_gb300.norm import group_norm_act
    x = torch.randn(2, 5, 16, device="cuda", requires_grad=True)
    f = lambda t: group_norm_act(t, 4, activation="silu")  # noqa: E731
    grad, = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            f(torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x)))
    for wrong in (lambda: torch.func.vmap(f)(x[None].detach()), lambda: torch.func.grad(lambda t: f(t).sum())(x.detach())):
        with pytest.raises(RuntimeError):
            wrong()


def amp_block(dtype):
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvBlock
    torch.manual_seed(0)
    block = WTConvBlock(24, levels=2, num_groups=4, device="cuda")
    x, t = torch.randn(3, 24, 20, 22, device="cuda"), torch.randn(3, 24, 20, 22, device="cuda")

    def run(x, dtype):
        x = x.detach().clone().requires_grad_()
        with torch.autocast("cuda", dtype=dtype or torch.float16, enabled=dtype is not None):
            y = block(x)
        return (y, *torch.autograd.grad((y.float() * t).sum(), [x, *block.parameters()]))

    return [n for n, _ in block.named_parameters()], run(x, None), run(x, dtype), run(x.to(dtype), dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_block_in_16_bits(ops, dtype):
    # Under autocast the pointwise products run in 16 bits; with a 16-bit input the
    # layer and the norms too.  Six roundings of 2^-11 (2^-8) on the way forward and
    # as many back, some of them amplified by the norms (weights near 1) and by sums
    # over 1320 pixels that partly cancel: 16 roundings are allowed.
    names, full, mixed, low = amp_block(dtype)
    tol = 16 * (2.0 ** -11 if dtype is torch.float16 else 2.0 ** -8)
    assert low[0].dtype is dtype and low[1].dtype is dtype and mixed[0].dtype is torch.float32
    for got in (mixed, low):
        for name, a, b in zip(["y", "x", *names], got, full):
            assert a.shape == b.shape and torch.isfinite(a).all()
            a, b = a.detach().double(), b.detach().double()
            assert float((a - b).norm() / b.norm()) <= tol, name
