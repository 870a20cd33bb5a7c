"""The gated channel mixer's modules: their gradients against plain torch in
float64, and all of them together, in training and in 8-bit inference.

Tolerances, derived before any run.  float32: the norm and the products are each
good to 1e-5 of their results' size (their own tests); a block chains six of them
forward and back, 1e-4 is asked.  8 bits: a rounding to e4m3 is off by 2^-4 at
most, about 0.026 in the root mean square; x and the two matrices have one each,
g and u therefore errors of 0.037 of their size, the product h of 0.07 with the
activation's slope (at most 1.1), and what the block adds to its input the same;
0.15 is asked of that part.
"""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def faults():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    yield
    assert blockops.wtconv_block_device_faults() == 0


def plain_norm(t, w, eps=1e-6):
    return t * (t.square().mean(-1, keepdim=True) + eps).rsqrt() * w


def plain_gated(x, gate, up, act):
    z = x @ gate.T
    z = torch.nn.functional.silu(z) if act == "silu" else torch.nn.functional.gelu(z) if act == "gelu" else z
    return z * (x @ up.T)


def close(a, b, tol):
    a, b = a.detach().double(), b.detach().double()
    assert a.shape == b.shape and float((a - b).norm()) <= tol * float(b.norm()), float((a - b).norm() / b.norm())


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_modules_against_autograd(act):
    from memory_bound_cnn_wtconv2d_gb300.mixer import GatedLinear, RMSNormAdd
    torch.manual_seed(3)
    norm, mix = RMSNormAdd(40, device="cuda"), GatedLinear(40, 72, act, device="cuda")
    with torch.no_grad():
        norm.weight.uniform_(0.5, 1.5)
    x, r = (torch.randn(2, 5, 7, 40, device="cuda", requires_grad=True) for _ in range(2))
    leaves = [x, r, norm.weight, mix.gate, mix.up]
    wide = [t.detach().double().requires_grad_() for t in leaves]

    def run(x, r, w, gate, up, plain):
        if plain:
            t = x + r
            return plain_gated(plain_norm(t, w), gate, up, act).sum(-1) + t.square().sum(-1)
        y, t = norm(x, r)
        return mix(y).sum(-1) + t.square().sum(-1)

    a, b = run(*leaves, False), run(*wide, True)
    close(a, b, 1e-5)
    for g, h in zip(torch.autograd.grad(a.sum(), leaves), torch.autograd.grad(b.sum(), wide)):
        assert g.dtype is F32
        close(g, h, 1e-4)
    alone = torch.autograd.grad(norm(x).square().sum(), [x, norm.weight])
    want = torch.autograd.grad(plain_norm(wide[0], wide[2]).square().sum(), [wide[0], wide[2]])
    for g, h in zip(alone, want):
        close(g, h, 1e-3)  # the norm's gradient of a norm: all but eps cancels
    y, t = norm(x, r)
    only, = torch.autograd.grad(t.sum(), x, retain_graph=True)  # the sum alone
    assert torch.equal(only, torch.ones_like(only))
    same = torch.autograd.grad(norm(x, x)[0].sum(), x)[0]  # one tensor in both places
    want = torch.autograd.grad(plain_norm(wide[0] + wide[0], wide[2]).sum(), wide[0])[0]
    close(same, want, 1e-4)


def test_frozen_and_broadcast(faults):
    from memory_bound_cnn_wtconv2d_gb300.mixer import GatedLinear, RMSNormAdd
    mix, norm = GatedLinear(32, 48, device="cuda"), RMSNormAdd(32, device="cuda")
    x = torch.randn(6, 32, device="cuda", requires_grad=True)
    mix.up.requires_grad_(False)
    mix(x).sum().backward()  # a gradient of stride 0
    assert mix.up.grad is None and mix.gate.grad is not None and x.grad is not None
    norm.weight.requires_grad_(False)
    norm(x).sum().backward()
    assert norm.weight.grad is None
    mix(x.detach()).sum().backward()
    with pytest.raises(RuntimeError):
        grad, = torch.autograd.grad(mix(x).square().sum(), x, create_graph=True)
        grad.sum().backward()


def test_the_block_and_a_step():
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvGatedBlock, block_optimizers
    from memory_bound_cnn_wtconv2d_gb300.clip import clip_grad_norm_
    torch.manual_seed(1)
    block = WTConvGatedBlock(24, levels=2, device="cuda")
    assert block.mix.hidden == 64
    x, t = torch.randn(3, 24, 20, 22, device="cuda", requires_grad=True), torch.randn(3, 24, 20, 22, device="cuda")
    y = block(x)
    params = list(block.parameters())
    grads = torch.autograd.grad((y * t).sum(), [x, *params])
    # the same around the same layer, in float64 behind it
    a = block.wtconv(x)
    wide = [p.detach().double().requires_grad_() for p in (block.norm.weight, block.mix.gate, block.mix.up, block.down.weight)]
    total = (a.double() + x.double()).permute(0, 2, 3, 1)
    z = (total + plain_gated(plain_norm(total, wide[0]), wide[1], wide[2], "silu") @ wide[3].T).permute(0, 3, 1, 2)
    close(y, z, 1e-5)
    names = {id(p): g for p, g in zip([x, *params], grads)}
    want = torch.autograd.grad((z * t.double()).sum(), [x, *wide, *block.wtconv.parameters()])
    got = [x, block.norm.weight, block.mix.gate, block.mix.up, block.down.weight, *block.wtconv.parameters()]
    for p, w in zip(got, want):
        close(names[id(p)], w, 1e-4)
    muon, adam = block_optimizers(block)
    assert len(muon.param_groups[0]["params"]) == 3
    for p, g in zip(params, grads[1:]):
        p.grad = g.clone()
    n = float(torch.stack([g.double().square().sum() for g in grads[1:]]).sum().sqrt())
    norm = clip_grad_norm_(block.parameters(), 0.5 * n)
    assert float(norm) == pytest.approx(n, rel=1e-5)
    for p, g in zip(params, grads[1:]):
        close(p.grad, g.double() * 0.5, 1e-5)
    before = [p.detach().clone() for p in params]
    muon.step()
    adam.step()
    assert all(not torch.equal(p, b) and torch.isfinite(p).all() for p, b in zip(params, before))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_the_block_in_16_bits(dtype):
    # roundings of 2^-11 (2^-8): five on the way forward, as many back, in sums over
    # 1320 pixels that partly cancel: 16 are allowed
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvGatedBlock
    torch.manual_seed(0)
    block = WTConvGatedBlock(24, levels=2, device="cuda")
    x, t = torch.randn(3, 24, 20, 22, device="cuda"), torch.randn(3, 24, 20, 22, device="cuda")

    def run(x, dtype):
        x = x.detach().clone().requires_grad_()
        with torch.autocast("cuda", dtype=dtype or F16, enabled=dtype is not None):
            y = block(x)
        return (y, *torch.autograd.grad((y.float() * t).sum(), [x, *block.parameters()]))

    full = run(x, None)
    for got in (run(x, dtype), run(x.to(dtype), dtype)):
        for a, b in zip(got, full):
            assert a.shape == b.shape and torch.isfinite(a).all()
            close(a, b, 16 * (2.0 ** -11 if dtype is F16 else 2.0 ** -8))


def test_inference_in_8_bits():
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvGatedBlock
    torch.manual_seed(2)
    block = WTConvGatedBlock(48, levels=2, device="cuda")
    x = torch.randn(2, 48, 28, 28, device="cuda")
    with torch.no_grad():
        want, base = block(x), x + block.wtconv(x)
        assert block.quantize_() is block and block.quantize_() is block
        got = block(x)
        close(got - base, want - base, 0.15)
        low = WTConvGatedBlock(48, levels=2, device="cuda").quantize_()
        low.load_state_dict(block.state_dict())
        assert torch.equal(low(x), got)
    with pytest.raises(RuntimeError, match="no_grad"):
        block(x)
    with pytest.raises(ValueError):
        WTConvGatedBlock(24, device="cuda").quantize_()


def test_a_captured_step_of_norm_product_and_clipping():
    from memory_bound_cnn_wtconv2d_gb300 import mixerops as ops
    torch.manual_seed(4)
    x, r, dh = (torch.randn(700, 64, device="cuda").to(BF16) for _ in range(3))
    gate, up, w = (torch.randn(64, 64, device="cuda") / 8).to(BF16), (torch.randn(64, 64, device="cuda") / 8).to(BF16), torch.rand(64, device="cuda")

    def step():
        y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=r)
        h = ops.wtconv_gated_fwd(y, gate, up)
        dy, dgate, dup = ops.wtconv_gated_bwd(dh, y, gate, up)
        dx, dw = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dh)
        norm = ops.wtconv_clip_grads([dgate, dup, dw], 1.0)
        return h, dx, dgate, dup, dw, norm

    graph = torch.cuda.CUDAGraph()
    step()
    with torch.cuda.graph(graph):
        captured = step()
    for scale in (1.0, 0.5, -2.0):
        x.copy_(torch.randn(700, 64, device="cuda") * scale)
        dh.copy_(torch.randn(700, 64, device="cuda") * scale)
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))


def test_two_streams_at_once():
    from memory_bound_cnn_wtconv2d_gb300 import mixerops as ops
    torch.manual_seed(5)
    sets = [[torch.randn(m, n, device="cuda").to(BF16) for m, n in ((3000, 200), (3000, 96), (200, 96), (200, 96))] for _ in range(2)]
    want = [ops.wtconv_gated_bwd(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(ops.wtconv_gated_bwd(*sets[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for g in got[i] for a, b in zip(g, want[i]))


def test_clipping_a_module():
    from memory_bound_cnn_wtconv2d_gb300.clip import clip_grad_norm_
    p, q, none = (torch.nn.Parameter(torch.randn(5, 3, device="cuda")) for _ in range(3))
    assert float(clip_grad_norm_([none], 1.0)) == 0
    p.grad, q.grad = torch.ones(5, 3, device="cuda"), torch.full((5, 3), 2.0, device="cuda")
    assert float(clip_grad_norm_([p, q, p, none], 1e9)) == pytest.approx(75 ** 0.5, rel=1e-6)
    assert torch.equal(p.grad, torch.ones_like(p))
    clip_grad_norm_(p, 0.0)
    assert not p.grad.any()
    q.grad[0, 0] = float("inf")
    before = q.grad.clone()
    with pytest.raises(RuntimeError):
        clip_grad_norm_([p, q], 1.0, error_if_nonfinite=True)
    assert torch.equal(q.grad, before)


def test_the_example_runs_with_gated_blocks():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, _ = mod.train(steps=3, channels=16, size=16, batch=8, log=None, gated=True)
    assert len(losses) == 3 and all(v == v for v in losses)
