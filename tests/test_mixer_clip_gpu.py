"""The global gradient norm and clipping by it, against float64.

Tolerances, derived before any run.  Squares of a few values (24 in a row at
most) are added in float32 (roundings of 2^-24 relative each, half of them on
average) and carried on in float64; the root halves a relative error and is
rounded once: 1e-6.  A clipped
element is one float32 product with a factor of that error and one rounding.
"""
import math

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import mixerops
    return mixerops


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def clipped64(ts, limit, eps=1e-6):
    f = min(1.0, limit / (norm64(ts) + eps))
    return [t.double() * f for t in ts]


def check(ts, want):
    for t, v in zip(ts, want):
        if not t.numel():
            continue
        half = 2.0 ** -24 if t.dtype is F32 else torch.finfo(t.dtype).eps / 2
        tiny = 2.0 ** -25 if t.dtype is F16 else 0.0
        assert float(((t.double() - v).abs() - (half + 3e-6) * v.abs() - tiny).max()) <= 0


LISTS = [[(1,)], [(5,), (3, 7)], [(96, 5, 5), (96,), (384, 96), (96, 384), (3, 384, 5, 5)], [(1000003,)], [(0,), (17,), (0, 3), (1,)],
         [(8192,), (8193,), (8191,)], [(2048, 1500)] * 3 + [(7,)] * 40, [(11,)] * 1500]


@pytest.mark.parametrize("dtype", [F32, F16, BF16, "mixed"])
@pytest.mark.parametrize("shapes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clipping(ops, shapes, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(len(shapes))
    types = [F32, F16, BF16]
    ts = [(0.1 * torch.randn(*s, generator=g, device="cuda")).to(types[i % 3] if dtype == "mixed" else dtype)
          for i, s in enumerate(shapes)]
    n = norm64(ts)
    got = ops.wtconv_grad_norm(ts)
    assert got.shape == () and got.dtype is F32 and float(got) == pytest.approx(n, rel=1e-6)
    before = [t.clone() for t in ts]
    assert torch.equal(ops.wtconv_clip_grads(ts, 2 * n + 1), got)  # below the limit
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    want = clipped64(ts, 0.37 * n)
    assert torch.equal(ops.wtconv_clip_grads(ts, 0.37 * n), got)
    check(ts, want)
    ops.wtconv_clip_grads(ts, 0.0)
    assert not any(t.any() for t in ts)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_views_of_one_buffer_at_any_offset(ops, dtype):
    flat = torch.randn(50021, device="cuda").to(dtype)
    sizes = [1, 2, 3, 5, 7, 4096, 9001, 13, 20000]
    keep = flat.clone()
    views, at = [], 3
    for s in sizes:
        views.append(flat[at:at + s])
        at += s + (s % 2)
    n = norm64(views)
    want = clipped64(views, 1.0)
    ops.wtconv_clip_grads(views, 1.0)
    check(views, want)
    assert float(ops.wtconv_grad_norm(flat[3:4])) == pytest.approx(norm64([flat[3:4]]), rel=1e-6)
    inside = torch.zeros(50021, dtype=torch.bool, device="cuda")
    at = 3
    for s in sizes:
        inside[at:at + s] = True
        at += s + (s % 2)
    assert torch.equal(flat[~inside], keep[~inside]) and n > 1


def test_other_orders_of_axes(ops):
    t = torch.randn(8, 16, 5, 3, device="cuda")
    views = [t.permute(0, 2, 3, 1), torch.randn(30, 40, device="cuda").t(), torch.randn(6, 1, 9, device="cuda").transpose(1, 2)]
    want = clipped64(views, 0.5)
    ops.wtconv_clip_grads(views, 0.5)
    check(views, want)


def test_values_whose_squares_leave_float32(ops):
    for size in (1e25, 3e36, 3e37, 1e-25, 1e-40):
        ts = [torch.randn(1000, device="cuda") * size, torch.randn(3, 3, device="cuda") * size]
        n = norm64(ts)
        got = float(ops.wtconv_grad_norm(ts))
        if n > torch.finfo(F32).max:  # 1000 values of 3e37: 9.6e38, which float32 does not have
            assert math.isinf(got)
            continue
        assert got == pytest.approx(n, rel=1e-6 if size > 1e-38 else 1e-2)
    ts = [torch.randn(1000, device="cuda").clamp(-3, 3) * 1e30]
    want = clipped64(ts, 2.0)
    ops.wtconv_clip_grads(ts, 2.0)
    check(ts, want)
    mixed = [torch.full((10,), 1e-30, device="cuda"), torch.full((10,), 1.0, device="cuda")]
    assert float(ops.wtconv_grad_norm(mixed)) == pytest.approx(math.sqrt(10), rel=1e-6)


def test_a_norm_that_is_not_finite(ops):
    ts = [torch.ones(100, device="cuda"), torch.ones(7, device="cuda", dtype=BF16)]
    ts[0][3] = float("inf")
    assert math.isinf(float(ops.wtconv_clip_grads(ts, 1.0)))
    assert torch.isnan(ts[0][3]) and not ts[0][4:].any() and not ts[1].any()
    ts = [torch.ones(100, device="cuda"), torch.ones(7, device="cuda", dtype=F16)]
    ts[1][0] = float("nan")
    assert math.isnan(float(ops.wtconv_clip_grads(ts, 1.0)))
    assert torch.isnan(ts[0]).all() and torch.isnan(ts[1]).all()


def test_same_bits_each_time_and_in_a_graph(ops):
    ts = [torch.randn(s, device="cuda") for s in ((2000, 700), (33,), (1, 5))]
    first = ops.wtconv_grad_norm(ts)
    assert all(torch.equal(ops.wtconv_grad_norm(ts), first) for _ in range(5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = ops.wtconv_clip_grads(ts, 1.0)
    for t in ts:
        t.mul_(3)
    want = clipped64(ts, 1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert float(a) == pytest.approx(3 * float(first), rel=1e-6)
    check(ts, want)


def test_a_given_norm_and_stream(ops):
    ts = [torch.randn(3000, device="cuda")]
    norm = torch.zeros((), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert ops.wtconv_grad_norm(ts, norm=norm, stream=side) is norm
    side.synchronize()
    assert float(norm) == pytest.approx(norm64(ts), rel=1e-6)


def test_autograd_learns_of_the_writing(ops):
    a = torch.randn(40, device="cuda", requires_grad=True)
    b = (a * 2).detach().requires_grad_()
    y = (b * b).sum()
    with torch.no_grad():
        ops.wtconv_clip_grads([b], 0.1)
    with pytest.raises(RuntimeError):
        y.backward()


def test_refusals(ops):
    t = torch.randn(64, device="cuda")
    for call in (lambda: ops.wtconv_grad_norm([]), lambda: ops.wtconv_grad_norm([t.cpu()]), lambda: ops.wtconv_grad_norm([t.double()]),
                 lambda: ops.wtconv_grad_norm([t[::2]]), lambda: ops.wtconv_grad_norm([t[:1].expand(5)]),
                 lambda: ops.wtconv_clip_grads([t, t], 1.0), lambda: ops.wtconv_clip_grads([t, t[10:20]], 1.0),
                 lambda: ops.wtconv_clip_grads([t], -1.0), lambda: ops.wtconv_clip_grads([t], float("nan")),
                 lambda: ops.wtconv_clip_grads([t], 1.0, eps=float("inf")), lambda: ops.wtconv_grad_norm([t], norm=t[:1]),
                 lambda: ops.wtconv_grad_norm([t], norm=t[0])):
        before = t.clone()
        with pytest.raises(ValueError):
            call()
        assert torch.equal(t, before)
    assert float(ops.wtconv_grad_norm([t, t])) == pytest.approx(math.sqrt(2) * norm64([t]), rel=1e-6)  # read only: allowed
