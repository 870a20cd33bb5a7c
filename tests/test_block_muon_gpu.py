"""Newton-Schulz orthogonalisation and the optimiser step, against float64.

Tolerances, derived before any run from a float64 simulation that rounds every
operand of the products as the library's header states.  Operands of 11
significand bits put 0.8e-3 to 1.8e-3 (relative 2-norm) on a full-rank result
of five steps, at most 3e-3 over the shapes tried; the result's own rounding
adds 2^-12 (float16) or 1.7e-3 (bfloat16): 5e-3 is asked.  Operands of 22 bits
are 2^11 times finer, and float32 sums of at most 8192 terms add a few 1e-6:
1e-5 is asked for float32.
"""
import math

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TOL = {F32: 1e-5, F16: 5e-3, BF16: 5e-3}
ABC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    yield blockops
    assert blockops.wtconv_block_device_faults() == 0


def ns64(g, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    x = g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + (b * s + c * s @ s) @ x
    return x.mT if tall else x


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm().clamp_min(1e-300))


def matrices(*shape, dtype=F32, seed=0, size=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


SHAPES = [(1, 1), (1, 7), (9, 1), (3, 5), (16, 16), (64, 64), (65, 63), (96, 384), (384, 96), (127, 129), (128, 128),
          (129, 130), (192, 768), (200, 1000), (257, 255), (333, 1201), (512, 512), (1000, 130), (640, 1030), (5, 4000), (128, 1024),
          (100, 1500), (2048, 60), (128, 2048), (700, 700), (1100, 1030), (900, 2300), (2100, 2050)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n", SHAPES)
def test_orthogonalize(ops, m, n, dtype):
    g = matrices(2, m, n, dtype=dtype, seed=m + n)
    out = ops.wtconv_orthogonalize(g)
    assert out.shape == g.shape and out.dtype == dtype and out.is_contiguous()
    for i in range(2):
        assert rel(out[i], ns64(g[i])) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("count,m,n", [(9, 384, 130), (3, 96, 100), (5, 300, 300), (70, 24, 40), (1, 1536, 1100)])
def test_stacks(ops, count, m, n, dtype):
    # different sizes in one stack: each matrix has its own norm
    g = matrices(count, m, n, dtype=F32, seed=count) * torch.logspace(-3, 3, count, device="cuda")[:, None, None]
    g = g.to(dtype)
    out = ops.wtconv_orthogonalize(g)
    for i in range(count):
        assert rel(out[i], ns64(g[i])) <= TOL[dtype], i


@pytest.mark.parametrize("steps", [0, 1, 2, 8])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_steps_and_coefficients(ops, steps, dtype):
    g = matrices(200, 310, dtype=dtype, seed=steps)
    for abc in (ABC, (1.5, -0.5, 0.0), (2.0, -1.5, 0.5)):
        out = ops.wtconv_orthogonalize(g, steps=steps, coefficients=abc)
        assert rel(out, ns64(g, steps, abc)) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_decaying_spectrum(ops, dtype):
    # singular values over three decades, as gradients have
    q = torch.linalg.qr(torch.randn(300, 300, dtype=torch.float64, device="cuda"))[0]
    v = torch.linalg.qr(torch.randn(700, 300, dtype=torch.float64, device="cuda"))[0]
    g = ((q * torch.logspace(0, -3, 300, device="cuda", dtype=torch.float64)) @ v.T).to(dtype)
    assert rel(ops.wtconv_orthogonalize(g), ns64(g)) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_low_rank(ops, dtype):
    # rank 3 of 160: the other directions hold rounding noise only, which both sides amplify
    g = (matrices(160, 3, seed=1, size=1.0) @ matrices(3, 250, seed=2, size=1.0)).to(dtype)
    g64, out = ns64(g), ops.wtconv_orthogonalize(g).double()
    u, s, v = torch.linalg.svd(g.double(), full_matrices=False)
    top = u[:, :3] @ (u[:, :3].T @ out @ v[:3].T) @ v[:3]
    want = u[:, :3] @ (u[:, :3].T @ g64 @ v[:3].T) @ v[:3]
    assert rel(top, want) <= TOL[dtype]


def test_zero_and_tiny(ops):
    z = torch.zeros(2, 40, 50, device="cuda")
    assert float(ops.wtconv_orthogonalize(z).abs().max()) == 0.0
    g = matrices(2, 40, 50, seed=3, size=1e-9)  # the norm is below eps
    g[1] = 0
    out = ops.wtconv_orthogonalize(g)
    assert rel(out[0], ns64(g[0])) <= 1e-5
    assert float(out[1].abs().max()) == 0.0


@pytest.mark.parametrize("size", [1e-12, 1e8])
def test_sizes_of_gradients(ops, size):
    g = matrices(60, 90, seed=4, size=size)
    assert rel(ops.wtconv_orthogonalize(g, eps=0.0), ns64(g, eps=0.0)) <= 1e-5


def test_one_large_entry(ops):
    # one entry holds nearly the whole norm
    g = matrices(150, 150, seed=5, size=1e-2)
    g[7, 9] = 10.0
    assert rel(ops.wtconv_orthogonalize(g), ns64(g)) <= 1e-5
    h = g.to(BF16)
    assert rel(ops.wtconv_orthogonalize(h), ns64(h)) <= 5e-3


def test_not_finite_stays_in_its_matrix(ops):
    g = matrices(3, 140, 200, seed=6)
    want = ops.wtconv_orthogonalize(g)
    g[1, 5, 6] = float("nan")
    out = ops.wtconv_orthogonalize(g)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert torch.isnan(out[1]).all()


def test_empty(ops):
    for shape in ((0, 4, 5), (2, 0, 5), (2, 4, 0)):
        g = torch.empty(shape, device="cuda")
        assert ops.wtconv_orthogonalize(g).shape == shape


@pytest.mark.parametrize("dtype", [F32, F16])
def test_rows_apart_and_odd_addresses(ops, dtype):
    for off, m, n in ((1, 70, 130), (3, 130, 70), (8, 64, 128)):
        wide = matrices(2, m, n + 24, dtype=dtype, seed=off)
        g = wide[:, :, off:off + n]
        out = torch.full((2, m, n + 5), 7.0, dtype=dtype, device="cuda")
        got = ops.wtconv_orthogonalize(g, out=out[:, :, 1:n + 1])
        assert got.data_ptr() == out[:, :, 1:].data_ptr()
        assert rel(got, ns64(g)) <= TOL[dtype]
        assert float((out[:, :, 0] - 7).abs().max()) == 0 and float((out[:, :, n + 1:] - 7).abs().max()) == 0


def test_same_from_run_to_run(ops):
    g = matrices(3, 500, 700, dtype=BF16, seed=7)
    want = ops.wtconv_orthogonalize(g)
    for _ in range(5):
        assert torch.equal(ops.wtconv_orthogonalize(g), want)


def test_given_workspace_stream_and_graph(ops):
    g = matrices(2, 300, 200, dtype=BF16, seed=8)
    want = ops.wtconv_orthogonalize(g)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.wtconv_orthogonalize(g, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(g)
    ops.wtconv_orthogonalize(g, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    src = g.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.wtconv_orthogonalize(src)
    for seed in (8, 9):
        h = matrices(2, 300, 200, dtype=BF16, seed=seed)
        src.copy_(h)
        graph.replay()
        assert torch.equal(out, ops.wtconv_orthogonalize(h))


def step64(w, g, b, lr, mu, nesterov, wd, scale):
    b = mu * b.double() + (1 - mu) * g.double()
    u = mu * b + (1 - mu) * g.double() if nesterov else b
    return (1 - lr * wd) * w.double() - lr * scale * ns64(u), b


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("count,m,n", [(1, 96, 384), (3, 384, 100), (2, 333, 201), (1, 7, 5), (1, 1, 1)])
def test_muon_step(ops, count, m, n, dtype, nesterov):
    # weight: the update is lr * scale * O with |O| known to TOL; relative to
    # the weight that is TOL * |update| / |weight|, plus one rounding
    w = matrices(count, m, n, dtype=dtype, seed=10, size=1 / math.sqrt(n))
    g = matrices(count, m, n, dtype=dtype, seed=11)
    b = matrices(count, m, n, seed=12)
    want_w, want_b = zip(*[step64(w[i], g[i], b[i], 0.02, 0.9, nesterov, 0.1, 1.3) for i in range(count)])
    before = w.double().clone()
    got = ops.wtconv_muon_step(w, g, b, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, scale=1.3)
    assert got is w
    rounding = {F32: 2.0 ** -23, F16: 2.0 ** -11, BF16: 2.0 ** -8}[dtype]
    for i in range(count):
        assert rel(b[i], want_b[i]) <= 1e-6
        update = float((want_w[i] - before[i]).norm())
        assert float((w[i].double() - want_w[i]).norm()) <= TOL[dtype] * update + rounding * float(want_w[i].norm())


def test_muon_step_lists_and_column_slices(ops):
    m, n = 100, 60
    ws = [matrices(m, n, seed=20 + i, size=0.1) for i in range(5)]
    gs = [matrices(m, n, seed=30 + i) for i in range(5)]
    bs = [torch.zeros(m, n, device="cuda") for _ in range(5)]
    want = [step64(w, g, b, 0.01, 0.95, True, 0.0, 1.0) for w, g, b in zip(ws, gs, bs)]
    ops.wtconv_muon_step(ws, gs, bs, lr=0.01)
    for w, b, (ww, bb) in zip(ws, bs, want):
        assert rel(w, ww) <= 1e-6 and rel(b, bb) <= 1e-6
    # the two halves of one fused matrix, side by side
    big, gbig, bbig = matrices(m, 2 * n, seed=40, size=0.1), matrices(m, 2 * n, seed=41), torch.zeros(m, 2 * n, device="cuda")
    want = [step64(big[:, k:k + n], gbig[:, k:k + n], bbig[:, k:k + n], 0.01, 0.95, True, 0.0, 1.0)[0] for k in (0, n)]
    halves = lambda t: [t[:, :n], t[:, n:]]  # noqa: E731
    ops.wtconv_muon_step(halves(big), halves(gbig), halves(bbig), lr=0.01)
    assert rel(big, torch.cat(want, 1)) <= 1e-6


def test_optimizer_matches_the_formula(ops):
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon, shape_scale
    torch.manual_seed(0)
    ps = [torch.nn.Parameter(torch.randn(s, device="cuda") * 0.1) for s in ((48, 20), (20, 48), (48, 20), (32, 16, 1, 1), (8, 8))]
    ref = [p.detach().double().clone() for p in ps]
    buf = [torch.zeros_like(r) for r in ref]
    opt = Muon(ps, lr=0.03, weight_decay=0.1)
    for it in range(3):
        for k, p in enumerate(ps):
            p.grad = None if k == 4 else torch.randn(p.shape, device="cuda", generator=None)
        for k, p in enumerate(ps):
            if p.grad is None:
                continue
            m = p.shape[0]
            g = p.grad.view(m, -1)
            w, b = step64(ref[k].view(m, -1), g, buf[k].view(m, -1), 0.03, 0.95, True, 0.1, shape_scale(m, g.shape[1]))
            ref[k], buf[k] = w.view(p.shape), b.view(p.shape)
        opt.step()
    for p, r in zip(ps, ref):
        assert rel(p.detach(), r) <= 1e-5
    state = opt.state_dict()
    again = Muon([torch.nn.Parameter(p.detach().clone()) for p in ps], lr=0.03, weight_decay=0.1)
    again.load_state_dict(state)
    assert torch.equal(again.state[again.param_groups[0]["params"][0]]["buffer"], opt.state[ps[0]]["buffer"])


def test_training_path(ops):
    # the small example, end to end: the loss falls well below chance (ln 6 = 1.79)
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(root, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, _ = mod.train(steps=40, channels=16, size=24, batch=48, log=None)
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-5:]) / 5 < 0.7 * losses[0]


def test_refusals(ops):
    g = matrices(2, 8, 12)
    f = ops.wtconv_orthogonalize
    bad = [lambda: f(g.cpu()), lambda: f(g[0, 0]), lambda: f(g.double()), lambda: f(g.mT), lambda: f(g, steps=-1),
           lambda: f(g, steps=65), lambda: f(g, steps=2.0), lambda: f(g, coefficients=(1.0, 2.0)),
           lambda: f(g, coefficients=(float("nan"), 0, 0)), lambda: f(g, coefficients=(17.0, 0, 0)), lambda: f(g, out=g),
           lambda: f(g, out=torch.empty(2, 8, 11, device="cuda")), lambda: f(g, out=torch.empty(2, 12, 8, device="cuda").mT),
           lambda: f(g, out=torch.empty(8, 12, device="cuda").expand(2, 8, 12)),
           lambda: f(g, workspace=torch.empty(10, dtype=torch.uint8))]
    w, b = matrices(2, 8, 12, seed=1), torch.zeros(2, 8, 12, device="cuda")
    s = ops.wtconv_muon_step
    bad += [lambda: s(w, g[:1], b, lr=0.1), lambda: s(w, g.half(), b, lr=0.1), lambda: s(w, g, b.half(), lr=0.1),
            lambda: s(w, w, b, lr=0.1), lambda: s(w, g, w, lr=0.1), lambda: s(w, g, g, lr=0.1), lambda: s([], [], [], lr=0.1),
            lambda: s(w, g, b, lr=float("inf")), lambda: s([w[0], w[0]], [g[0], g[1]], [b[0], b[1]], lr=0.1),
            lambda: s([w[0], w[1][:4]], [g[0], g[1]], [b[0], b[1]], lr=0.1)]
    keep = [t.clone() for t in (g, w, b)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert all(torch.equal(p, q) for p, q in zip(keep, (g, w, b)))
    from memory_bound_cnn_wtconv2d_gb300 import wtconv
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    with pytest.raises(wtconv.WtconvError) as e:
        f(matrices(2, 200, 300), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == wtconv.WTCONV_ERR_WORKSPACE
    with pytest.raises(wtconv.WtconvError) as e:
        f(g, eps=-1.0)
    assert e.value.status == wtconv.WTCONV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(3))])
    with pytest.raises(ValueError):
        Muon([torch.nn.Parameter(torch.zeros(3, 3))], momentum=1.0)


def test_workspace_belongs_to_the_given_stream(ops):
    # the stream is held up while the caller's stream reuses all memory that is free to it
    g = matrices(2, 300, 200, dtype=BF16, seed=31)
    want = ops.wtconv_orthogonalize(g)
    need = ops._ns_desc(ops._Stack(g, "g"), 2, 5, ops.NS_COEFFICIENTS, 1e-7)[1]
    assert need > 0
    for handle in (False, True):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
        got = ops.wtconv_orthogonalize(g, stream=s.cuda_stream if handle else s)
        for _ in range(50):
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)
        s.synchronize()
        assert torch.equal(want, got)


@pytest.mark.parametrize("m,n", [(275, 3176), (3176, 275), (300, 9000), (520, 1601)])
def test_long_rows(ops, m, n):
    # the diagonal of X X^T is a sum of n squares, of which every addition loses a little
    g = matrices(m, n, seed=m + n)
    assert rel(ops.wtconv_orthogonalize(g), ns64(g)) <= TOL[F32]
