"""Group norm with an activation on channels-last activations, against a plain
float64 implementation.

Tolerances, derived before any run.  float32: a value of y or dx comes from a
handful of float32 operations on numbers of the size of xhat (at most sqrt of
the group's size, in practice below 10) and from statistics whose relative
error is a few units of 2^-24: 2e-6 of the result's root mean square per
operation bounds it, 1e-5 relative 2-norm is asked.  16-bit results: one
rounding to nearest more, 2^-11 (float16) or 2^-8 (bfloat16) relative at most,
so half of that again is allowed.  Parameter gradients are float32 sums of n
terms in blocks, relative to the root of the sum of squares of their terms:
1e-5.
"""
import math

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TOL = {F32: 1e-5, F16: 1.5 * 2.0 ** -11, BF16: 1.5 * 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


def inputs(shape, dtype, seed=0, shift=0.3, affine=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    C = shape[-1]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(*shape) * (0.5 + torch.rand(C, generator=g, device="cuda")) + shift * r(C)).to(dtype)
    dy = r(*shape).to(dtype)
    return x, dy, (1 + 0.2 * r(C) if affine else None), (0.2 * r(C) if affine else None)


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def grad64(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def forward64(x, G, w, b, eps, act):
    N, C = x.shape[0], x.shape[-1]
    x = x.double().reshape(N, -1, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    z = (x - mean) * rstd * (1.0 if w is None else w.double().view(G, -1)) + (0.0 if b is None else b.double().view(G, -1))
    return act64(z, act), mean.view(N, G), rstd.view(N, G)


def backward64(dy, x, G, w, b, eps, act):
    N, C = x.shape[0], x.shape[-1]
    x = x.double().reshape(N, -1, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    w = torch.ones(G, C // G, dtype=torch.float64, device=x.device) if w is None else w.double().view(G, -1)
    b = torch.zeros_like(w) if b is None else b.double().view(G, -1)
    xh = (x - mean) * rstd
    dz = dy.double().reshape(x.shape) * grad64(xh * w + b, act)
    dxh = dz * w
    dx = rstd * (dxh - dxh.mean((1, 3), keepdim=True) - xh * (dxh * xh).mean((1, 3), keepdim=True))
    return dx, (dz * xh).sum((0, 1)).view(C), dz.sum((0, 1)).view(C), dz, dz * xh


def rel(a, b):
    a, b = a.double().reshape(-1), b.double().reshape(-1)
    return float((a - b).norm() / b.norm().clamp_min(1e-300))


def check_forward(ops, x, G, w, b, act, eps=1e-5, dtype=None, **kw):
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, G, w, b, eps=eps, activation=act, **kw)
    ry, rm, rr = forward64(x, G, w, b, eps, act)
    assert y.shape == x.shape and y.is_contiguous() and y.dtype == x.dtype
    assert rel(y, ry) <= TOL[x.dtype]
    # element by element too, against the largest value of the result
    worst = (y.double().reshape(ry.shape) - ry).abs().max() / ry.abs().max()
    assert float(worst) <= 2 * TOL[x.dtype]
    scale = float(1 / rr.min())
    assert float((mean.double() - rm).abs().max()) <= 1e-6 * max(scale, float(rm.abs().max()))
    assert rel(rstd, rr) <= 1e-5
    return y, mean, rstd


def check_backward(ops, dy, x, G, w, b, act, eps=1e-5, **kw):
    _, mean, rstd = ops.wtconv_gn_act_fwd(x, G, w, b, eps=eps, activation=act)
    dx, dw, db = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, G, w, b, activation=act, **kw)
    rdx, rdw, rdb, t0, t1 = backward64(dy, x, G, w, b, eps, act)
    assert dx.shape == x.shape and dx.dtype == x.dtype
    # dx is a difference of terms of the size of rstd * w * dz: where they
    # cancel (few values a group), its error is relative to them
    terms = float((rdx.norm() ** 2 + (0.1 * float(rstd.double().mean()) * t0.norm()) ** 2).sqrt())
    assert float((dx.double().reshape(rdx.shape) - rdx).norm()) <= TOL[x.dtype] * max(terms, 1e-30)
    n0 = t0.square().sum((0, 1)).sqrt().norm()
    n1 = t1.square().sum((0, 1)).sqrt().norm()
    assert float((db.double() - rdb).norm() / n0.clamp_min(1e-300)) <= 1e-5
    assert float((dw.double() - rdw).norm() / n1.clamp_min(1e-300)) <= 1e-5
    return dx, dw, db


SHAPES = [((2, 8, 8, 32), 4), ((1, 1, 1, 8), 2), ((3, 5, 7, 30), 6), ((2, 9, 11, 45), 5), ((1, 49, 768), 32),
          ((2, 56, 56, 96), 32), ((4, 14, 14, 384), 32), ((3, 33, 7), 7), ((2, 13, 1024), 1), ((1, 3, 2056), 8),
          ((5, 37, 53, 90), 6), ((1, 200, 201, 12), 3), ((2, 120, 120, 64), 8), ((70, 6, 6, 16), 4), ((2, 4, 4, 8192), 64),
          ((1, 100, 100, 5), 5), ((2, 64, 4096), 2), ((3, 300, 40), 1)]


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shape,G", SHAPES)
def test_forward(ops, shape, G, dtype, act):
    x, _, w, b = inputs(shape, dtype, seed=len(shape) + shape[-1])
    check_forward(ops, x, G, w, b, act)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("shape,G", [s for s in SHAPES if math.prod(s[0][1:-1]) * s[0][-1] // s[1] > 8])
def test_backward(ops, shape, G, dtype, act):
    x, dy, w, b = inputs(shape, dtype, seed=len(shape) + shape[-1])
    check_backward(ops, dy, x, G, w, b, act)


@pytest.mark.parametrize("which", ["neither", "weight", "bias"])
def test_optional_parameters(ops, which):
    x, dy, w, b = inputs((2, 6, 6, 24), F32, seed=3)
    w, b = (w if which == "weight" else None), (b if which == "bias" else None)
    check_forward(ops, x, 3, w, b, "silu")
    check_backward(ops, dy, x, 3, w, b, "silu")


def test_one_value_per_group(ops):
    # a group of one value: xhat is 0, y = act(bias), and nothing flows back to x
    x, dy, w, b = inputs((2, 1, 1, 6), F32, seed=4)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 6, w, b, activation="gelu")
    assert torch.equal(mean, x.view(2, 6))
    assert rel(y, act64(b.double(), "gelu").expand(2, 6)) <= 1e-6
    dx, dw, db = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 6, w, b, activation="gelu")
    scale = float(rstd.max()) * float(dy.abs().max())
    assert float(dx.abs().max()) <= 1e-5 * scale
    assert float(dw.abs().max()) == 0.0


@pytest.mark.parametrize("shape,G", [((2, 16, 16, 32), 4), ((2, 120, 120, 64), 8), ((2, 10, 10, 45), 5)])
def test_mean_far_from_zero(ops, shape, G):
    # mean / deviation = 4096: a sum of squares in float32 would lose 2^24 of
    # its digits.  x is exact to 2^-24 * 4096 of a deviation, the statistics'
    # pivots and merges lose a few of those: 1e-3 leaves an order of magnitude.
    x, _, w, b = inputs(shape, F32, seed=5, shift=0.0)
    x = x + 4096.0
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, G, w, b)
    ry, rm, rr = forward64(x, G, w, b, 1e-5, "none")
    assert rel(y, ry) <= 1e-3
    assert rel(rstd, rr) <= 1e-3
    assert rel(mean, rm) <= 1e-6


def test_one_outlier_first(ops):
    # the value a pivot is taken from is 1000 deviations off
    x, _, w, b = inputs((1, 40, 40, 16), F32, seed=6)
    x[0, 0, 0, :] = 1000.0
    check_forward(ops, x, 2, w, b, "none")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_constant_input(ops, dtype):
    # no variance: rstd = 1 / sqrt(eps), y = act(bias)
    x = torch.full((2, 9, 9, 16), 0.75, dtype=dtype, device="cuda")
    _, _, w, b = inputs((2, 9, 9, 16), dtype, seed=7)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 4, w, b, eps=1e-5, activation="silu")
    assert torch.equal(mean, torch.full_like(mean, 0.75))
    assert rel(rstd, torch.full_like(rstd, 1e-5 ** -0.5)) <= 1e-6
    assert rel(y, act64(b.double(), "silu").expand(x.shape)) <= TOL[dtype]


def test_large_activations_saturate(ops):
    # activations far out: silu and gelu go to 0 and to z, without overflow
    x = torch.linspace(-1, 1, 64, device="cuda").view(1, 8, 8, 1).repeat(1, 1, 1, 4).contiguous()
    w = torch.tensor([1.0, 30.0, 200.0, 1e4], device="cuda")
    b = torch.zeros(4, device="cuda")
    for act in ("silu", "gelu"):
        check_forward(ops, x, 1, w, b, act)
        _, mean, rstd = ops.wtconv_gn_act_fwd(x, 1, w, b, activation=act)
        dx, dw, db = ops.wtconv_gn_act_bwd(torch.ones_like(x), x, mean, rstd, 1, w, b, activation=act)
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_not_finite_values_stay_in_their_group(ops):
    x, dy, w, b = inputs((3, 12, 12, 32), F32, seed=8)
    clean, _, _ = ops.wtconv_gn_act_fwd(x, 4, w, b, activation="silu")
    x[1, 3, 4, 9] = float("nan")
    x[2, 0, 0, 31] = float("inf")
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 4, w, b, activation="silu")
    v, c = y.view(3, 144, 4, 8), clean.view(3, 144, 4, 8)
    for n, g in ((n, g) for n in range(3) for g in range(4)):
        if (n, g) in ((1, 1), (2, 3)):
            assert torch.isnan(v[n, :, g]).all()
        else:
            assert torch.equal(v[n, :, g], c[n, :, g])
    dx, _, _ = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 4, w, b, activation="silu")
    d = dx.view(3, 144, 4, 8)
    for n, g in ((n, g) for n in range(3) for g in range(4)):
        assert torch.isfinite(d[n, :, g]).all() == ((n, g) not in ((1, 1), (2, 3)))


def test_empty(ops):
    w, b = torch.ones(8, device="cuda"), torch.zeros(8, device="cuda")
    for shape in ((0, 4, 4, 8), (2, 0, 4, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = ops.wtconv_gn_act_fwd(x, 2, w, b)
        assert y.shape == x.shape and mean.shape == (shape[0], 2)
        assert float(mean.abs().sum()) == 0.0
        dw, db = torch.full((8,), 7.0, device="cuda"), torch.full((8,), 7.0, device="cuda")
        dx, dw, db = ops.wtconv_gn_act_bwd(x, x, mean, rstd, 2, w, b, dweight=dw, dbias=db)
        assert float(dw.abs().sum()) == 0.0 and float(db.abs().sum()) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,G", [((3, 6, 5, 24), 4), ((2, 64, 64, 48), 8), ((2, 20, 30, 30), 3)])
def test_slices_of_wider_tensors(ops, shape, G, dtype):
    # channels out of a wider tensor, at aligned and odd offsets; samples apart
    N, H, W, C = shape
    for off, wide in ((8, C + 16), (3, C + 7), (0, C + 1)):
        big, bigd, w, b = inputs((2 * N, H, W, wide), dtype, seed=off)
        x, dy = big[::2, :, :, off:off + C], bigd[::2, :, :, off:off + C]
        w, b = w[off:off + C].clone(), b[off:off + C].clone()
        y, mean, rstd = ops.wtconv_gn_act_fwd(x, G, w, b, activation="silu")
        ry, _, _ = forward64(x, G, w, b, 1e-5, "silu")
        assert rel(y, ry) <= TOL[dtype]
        dx, dw, db = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, G, w, b, activation="silu")
        rdx, rdw, rdb, _, _ = backward64(dy, x, G, w, b, 1e-5, "silu")
        assert rel(dx, rdx) <= 2 * TOL[dtype]
        assert rel(db, rdb) <= 1e-4 and rel(dw, rdw) <= 1e-4


@pytest.mark.parametrize("dtype", [F32, F16])
def test_unaligned_base(ops, dtype):
    # one element past a 16-byte boundary, in and out
    N, S, C = 2, 50, 64
    buf = torch.randn(N * S * C + 1, device="cuda").to(dtype)
    x = buf[1:].view(N, S, C)
    out = torch.empty(N * S * C + 1, dtype=dtype, device="cuda")[1:].view(N, S, C)
    _, dy, w, b = inputs((N, S, C), dtype, seed=9)
    y, _, _ = check_forward(ops, x, 8, w, b, "gelu", y=out)
    assert y.data_ptr() == out.data_ptr()
    check_backward(ops, dy, x, 8, w, b, "gelu", dx=torch.empty_like(out))


def test_broadcast_rows(ops):
    # every pixel of a sample the same row of memory (stride 0)
    row, _, w, b = inputs((2, 1, 16), F32, seed=10)
    x = row.expand(2, 30, 16)
    y, _, _ = ops.wtconv_gn_act_fwd(x, 2, w, b)
    ry, _, _ = forward64(x, 2, w, b, 1e-5, "none")
    assert rel(y, ry) <= 1e-5


def test_same_from_run_to_run_and_into_given_buffers(ops):
    x, dy, w, b = inputs((7, 40, 40, 48), BF16, seed=11)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 8, w, b, activation="silu")
    g = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 8, w, b, activation="silu")
    y2, mean2, rstd2 = torch.empty_like(y), torch.empty_like(mean), torch.empty_like(rstd)
    dirty = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    ops.wtconv_gn_act_fwd(x, 8, w, b, activation="silu", y=y2, mean=mean2, rstd=rstd2, workspace=dirty)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    for _ in range(3):
        dirty.fill_(255)
        again = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 8, w, b, activation="silu", workspace=dirty)
        assert all(torch.equal(p, q) for p, q in zip(g, again))


def test_another_stream_and_a_graph(ops):
    x, dy, w, b = inputs((4, 28, 28, 96), F16, seed=12)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 32, w, b, activation="gelu")
    g = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 32, w, b, activation="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, _, _ = ops.wtconv_gn_act_fwd(x, 32, w, b, activation="gelu", y=torch.empty_like(y), stream=s)
    s.synchronize()
    assert torch.equal(y, y2)
    xs, dys = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, mg, rg = ops.wtconv_gn_act_fwd(xs, 32, w, b, activation="gelu")
        gg = ops.wtconv_gn_act_bwd(dys, xs, mg, rg, 32, w, b, activation="gelu")
    for seed in (12, 13):
        a, d, _, _ = inputs((4, 28, 28, 96), F16, seed=seed)
        xs.copy_(a)
        dys.copy_(d)
        graph.replay()
        ya, ma, ra = ops.wtconv_gn_act_fwd(a, 32, w, b, activation="gelu")
        ga = ops.wtconv_gn_act_bwd(d, a, ma, ra, 32, w, b, activation="gelu")
        assert torch.equal(yg, ya) and all(torch.equal(p, q) for p, q in zip(gg, ga))


def test_offsets_beyond_32_bits(ops):
    # rows 2^24 elements apart: the last lie 4.3 G elements (8.6 GB) behind the first
    rows, C = 260, 8
    big = torch.empty((rows - 1) * (1 << 24) + C, dtype=BF16, device="cuda")
    x = torch.as_strided(big, (1, rows, C), (big.numel(), 1 << 24, 1))
    small, dy, w, b = inputs((1, rows, C), BF16, seed=14)
    x.copy_(small)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 2, w, b, activation="silu")
    want, m, r = ops.wtconv_gn_act_fwd(small, 2, w, b, activation="silu")
    assert torch.equal(y, want)
    got = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 2, w, b, activation="silu")
    ref = ops.wtconv_gn_act_bwd(dy, small, m, r, 2, w, b, activation="silu")
    assert all(torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gradients_against_differences(ops, act):
    # central differences of the float64 forward in random directions, against
    # the module's gradients of the same scalar.  Differences with step h err
    # by h^2 times third derivatives (1e-8 here); the kernels by float32.
    from memory_bound_cnn_wtconv2d_gb300.norm import GroupNormAct
    torch.manual_seed(15)
    m = GroupNormAct(3, 12, activation=act, device="cuda")
    with torch.no_grad():
        m.weight.add_(0.3 * torch.randn_like(m.weight))
        m.bias.add_(0.3 * torch.randn_like(m.bias))
    x = torch.randn(2, 4, 5, 12, device="cuda", requires_grad=True)
    t = torch.randn(2, 4, 5, 12, device="cuda")
    (m(x) * t).sum().backward()
    f = lambda x, w, b: float((forward64(x, 3, w, b, m.eps, act)[0].view(x.shape) * t.double()).sum())  # noqa: E731
    base = [x.detach().double(), m.weight.detach().double(), m.bias.detach().double()]
    h = 1e-4
    for k, grad in enumerate((x.grad, m.weight.grad, m.bias.grad)):
        for _ in range(4):
            v = torch.randn_like(base[k])
            up, down = list(base), list(base)
            up[k], down[k] = base[k] + h * v, base[k] - h * v
            slope = (f(*up) - f(*down)) / (2 * h)
            got = float((grad.double() * v).sum())
            size = float(grad.double().norm() * v.norm())
            assert abs(got - slope) <= 1e-5 * size + 1e-6


def test_module_takes_gradients_of_any_layout(ops):
    from memory_bound_cnn_wtconv2d_gb300.norm import GroupNormAct
    m = GroupNormAct(4, 16, activation="silu", device="cuda")
    x = torch.randn(2, 5, 6, 16, device="cuda", requires_grad=True)
    m(x).permute(0, 3, 1, 2).mean().backward()  # a broadcast upstream gradient
    a = x.grad.clone()
    x.grad = None
    y = m(x)
    y.backward(torch.full_like(y, 1.0 / y.numel()))
    assert torch.equal(a, x.grad)


def test_module_without_parameters_and_partial_gradients(ops):
    from memory_bound_cnn_wtconv2d_gb300.norm import GroupNormAct
    m = GroupNormAct(4, 16, affine=False, activation="gelu", device="cuda")
    x = torch.randn(2, 5, 6, 16, device="cuda", requires_grad=True)
    m(x).square().sum().backward()
    assert torch.isfinite(x.grad).all() and not list(m.parameters())
    m = GroupNormAct(4, 16, activation="gelu", device="cuda")
    m.weight.requires_grad_(False)
    m(x.detach()).sum().backward()
    assert m.weight.grad is None and m.bias.grad is not None


def test_refusals(ops):
    x = torch.randn(2, 4, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    f = ops.wtconv_gn_act_fwd
    bad = [
        lambda: f(x.cpu(), 4), lambda: f(x, 5), lambda: f(x, 0), lambda: f(x, 4, activation="relu"),
        lambda: f(x.double(), 4), lambda: f(x[0, 0], 4), lambda: f(x, 4, w[:8]), lambda: f(x, 4, w.half()),
        lambda: f(x, 4, w.cpu()), lambda: f(x.transpose(1, 2), 4), lambda: f(x, 4, y=torch.empty(2, 4, 15, device="cuda")),
        lambda: f(x, 4, y=x), lambda: f(x, 4, mean=torch.empty(2, 3, device="cuda")),
        lambda: f(torch.randn(2, 4, 5, 16, device="cuda").transpose(1, 2), 4),
        lambda: f(x, 4, y=torch.empty_like(x), workspace=torch.empty(256, dtype=torch.uint8)),
    ]
    y, mean, rstd = f(x, 4, w)
    g = ops.wtconv_gn_act_bwd
    bad += [
        lambda: g(x[:1], x, mean, rstd, 4), lambda: g(x.half(), x, mean, rstd, 4), lambda: g(x, x, mean[:, :2], rstd, 4),
        lambda: g(x, x, None, rstd, 4), lambda: g(x, x, mean, rstd, 4, dx=x), lambda: g(x, x, mean, rstd, 3),
        lambda: g(x, x, mean, rstd, 4, dweight=w, weight=w),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    from memory_bound_cnn_wtconv2d_gb300 import wtconv
    with pytest.raises(wtconv.WtconvError) as e:
        f(x, 4, w, eps=-1.0)
    assert e.value.status == wtconv.WTCONV_ERR_INVALID_ARG
    with pytest.raises(wtconv.WtconvError) as e:
        g(x, x, mean, rstd, 4, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == wtconv.WTCONV_ERR_WORKSPACE


def test_allocations_belong_to_the_given_stream(ops):
    # the stream is held up while the caller's stream reuses all memory that is free to it
    x, dy, w, b = inputs((8, 64, 64, 64), BF16, seed=21)
    y, mean, rstd = ops.wtconv_gn_act_fwd(x, 8, w, b, activation="silu")
    want = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 8, w, b, activation="silu")
    need = ops._gn_layout(x, dy, 8, 0.0, "silu").ws
    assert need > 0
    for handle in (False, True):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = ops.wtconv_gn_act_bwd(dy, x, mean, rstd, 8, w, b, activation="silu", stream=s.cuda_stream if handle else s)
        for _ in range(50):
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
