"""The gated product and its gradients against a plain float64 implementation.

Tolerances, derived before any run.  Forward: products of 16-bit operands are
exact, sums are float32 (float32 operands keep 24 bits), so g and u are off by
a few 2^-24 of |x||w| times the root of the length, below 1e-5 of their size up
to the lengths here; h then takes one rounding (16 bits: eps / 2 relative).
Backward: dg and du are held in the type (eps / 2 relative each, independent of
one another), so a sum over them is off by at most eps / 2 of the root of the
sum of squares of its terms times a normal deviate's spread of 0.6, of which
ten (six deviations) are allowed; then one rounding.  In float32 1e-5 stands for
both.
"""
import math

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build, wtconv

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ACTS = ["none", "silu", "gelu"]


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops, mixerops
    yield mixerops
    assert blockops.wtconv_block_device_faults() == 0


def half(dtype):
    return 2.0 ** -24 if dtype is F32 else torch.finfo(dtype).eps / 2


def inputs(M, C, H, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(M, H).to(dtype), r(M, C).to(dtype), (r(H, C) * 1.5 / math.sqrt(C)).to(dtype), (r(H, C) / math.sqrt(C)).to(dtype)


def act64(z, act):
    return z if act == "none" else torch.nn.functional.silu(z) if act == "silu" else z * torch.special.ndtr(z)


def grad64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def near(got, want, dtype, size):
    """One rounding of the value, and what the sums leave (`size`, by value)."""
    off = (got.double() - want).abs() - half(dtype) * want.abs() * 1.01 - size
    if dtype is F16:
        off = off - 2.0 ** -25
    assert got.shape == want.shape and got.dtype == dtype
    assert not want.numel() or float(off.max()) <= 0, (float(off.max()), float(want.abs().max()))


def check_forward(h, x, gate, up, act, scale=1.0):
    x, gate, up = x.double(), gate.double(), up.double()
    g, u = x @ gate.T, x @ up.T
    # what an error of 1e-5 of |x||w| leaves on the product of act(g) and u
    n = x.norm(dim=-1, keepdim=True) * 1e-5
    dg, du = n * gate.norm(dim=1), n * up.norm(dim=1)
    near(h, act64(g, act) * u, h.dtype, 1.2 * (dg * (u.abs() + du) + du * g.abs()) * scale)


def check_backward(got, dh, x, gate, up, act, dtype):
    dh, x, gate, up = (t.double() for t in (dh, x, gate, up))
    g, u = x @ gate.T, x @ up.T
    dg, du = dh * u * grad64(g, act), dh * act64(g, act)
    each = (10 * half(dtype) if dtype is not F32 else 0.0) * 0.6 + 1e-5
    root = lambda a, b: ((a * a) @ (b * b)).sqrt()  # noqa: E731
    # the float32 sums behind g and u leave errors of their own size on dg and du
    n = x.norm(dim=-1, keepdim=True) * 1e-5
    eg = dh.abs() * 1.2 * (n * up.norm(dim=1) + (u.abs() + n) * n * gate.norm(dim=1))
    eu = dh.abs() * 1.2 * n * gate.norm(dim=1)
    dx, dgate, dup = got
    if dx is not None:
        near(dx, dg @ gate + du @ up, dtype,
             each * (root(dg, gate) + root(du, up)) + 4 * (root(eg, gate) + root(eu, up)))
    if dgate is not None:
        near(dgate, dg.T @ x, dtype, each * root(dg.T, x) + 4 * root(eg.T, x))
        near(dup, du.T @ x, dtype, each * root(du.T, x) + 4 * root(eu.T, x))


SHAPES = [(1, 1, 1), (1, 768, 2048), (2, 64, 64), (5, 33, 17), (8, 96, 256), (9, 96, 256), (49, 768, 200), (100, 90, 237),
          (127, 64, 128), (128, 128, 128), (129, 72, 130), (300, 96, 384), (513, 200, 1000), (1000, 1000, 24), (2000, 8, 700),
          (257, 1500, 333), (4099, 40, 56), (700, 384, 1024), (20000, 96, 100)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C,H", SHAPES)
def test_forward(ops, M, C, H, dtype):
    _, x, gate, up = inputs(M, C, H, dtype, M + H)
    for act in ACTS:
        check_forward(ops.wtconv_gated_fwd(x, gate, up, activation=act), x, gate, up, act)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C,H", SHAPES)
def test_backward(ops, M, C, H, dtype):
    dh, x, gate, up = inputs(M, C, H, dtype, M + C)
    act = ACTS[(M + C + H) % 3]
    got = ops.wtconv_gated_bwd(dh, x, gate, up, activation=act)
    check_backward(got, dh, x, gate, up, act, dtype)
    again = ops.wtconv_gated_bwd(dh, x, gate, up, activation=act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    dx, none, none2 = ops.wtconv_gated_bwd(dh, x, gate, up, activation=act, need_dweights=False)
    assert none is none2 is None and torch.equal(dx, got[0])
    none, dgate, dup = ops.wtconv_gated_bwd(dh, x, gate, up, activation=act, need_dx=False)
    assert none is None and torch.equal(dgate, got[1]) and torch.equal(dup, got[2])


@pytest.mark.parametrize("act", ACTS)
def test_gradients_by_differences(ops, act):
    dh, x, gate, up = inputs(7, 40, 24, F32)
    grads = ops.wtconv_gated_bwd(dh, x, gate, up, activation=act)
    loss = lambda x, gate, up: float((act64(x @ gate.T, act) * (x @ up.T) * dh.double()).sum())  # noqa: E731
    vs = [t.double() for t in (x, gate, up)]
    for k, grad in enumerate(grads):
        d = torch.randn_like(vs[k])
        step = 1e-5
        plus, minus = ([v + s * step * d if i == k else v for i, v in enumerate(vs)] for s in (1, -1))
        want = (loss(*plus) - loss(*minus)) / (2 * step)
        assert float((grad.double() * d).sum()) == pytest.approx(want, rel=1e-4, abs=1e-4)


def quantised(ops, M, C, H, seed):
    _, x, gate, up = inputs(M, C, H, F32, seed)
    return [*ops.wtconv_quantize_rows(x), *ops.wtconv_quantize_rows(gate), *ops.wtconv_quantize_rows(up)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C,H", [(1, 16, 1), (1, 768, 2048), (3, 32, 40), (8, 96, 256), (9, 112, 256), (130, 128, 130), (128, 256, 128),
                                   (257, 1504, 333), (1000, 48, 1000), (5000, 384, 512)])
def test_8_bit_operands(ops, M, C, H, dtype):
    x, xs, gate, gs, up, us = quantised(ops, M, C, H, M)
    d = lambda q, s: q.double() * s.double()[:, None]  # noqa: E731
    for act in ACTS:
        h = ops.wtconv_gated_q8(x, xs, gate, gs, up, us, activation=act, dtype=dtype)
        assert h.dtype is dtype
        check_forward(h, d(x, xs), d(gate, gs), d(up, us), act)


@pytest.mark.parametrize("dtype", TYPES)
def test_slices_and_leading_axes(ops, dtype):
    for a, b, H in ((0, 96, 128), (64, 160, 72), (1, 97, 64), (8, 75, 100)):
        wide = torch.randn(2, 9, 11, 200, device="cuda").to(dtype)
        weights = (torch.randn(2 * H + 3, 200, device="cuda") / 10).to(dtype)
        hid = torch.randn(2, 9, 11, H + 40, device="cuda").to(dtype)
        x, gate, up, dh = wide[..., a:b], weights[:H, a:b], weights[H + 3:, a:b], hid[..., 3:3 + H]
        h = ops.wtconv_gated_fwd(x, gate, up)
        assert h.shape == (2, 9, 11, H) and h.is_contiguous()
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        check_forward(flat(h), flat(x), gate, up, "silu")
        dx, dgate, dup = ops.wtconv_gated_bwd(dh, x, gate, up)
        check_backward((flat(dx), dgate, dup), flat(dh), flat(x), gate, up, "silu", dtype)
    row = wide[0, 0, 0, a:b]
    check_forward(ops.wtconv_gated_fwd(row, gate, up)[None], row[None], gate, up, "silu")


@pytest.mark.parametrize("dtype", TYPES)
def test_empty(ops, dtype):
    x = torch.empty(0, 3, 64, device="cuda", dtype=dtype)
    gate, up = torch.randn(2, 40, 64, device="cuda").to(dtype).unbind()
    assert ops.wtconv_gated_fwd(x, gate, up).shape == (0, 3, 40)
    dx, dgate, dup = ops.wtconv_gated_bwd(torch.empty(0, 3, 40, device="cuda", dtype=dtype), x, gate, up)
    assert dx.shape == x.shape and not dgate.any() and not dup.any()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 200])
def test_a_row_that_is_not_finite_stays_alone(ops, M, dtype):
    _, x, gate, up = inputs(M, 96, 200, dtype)
    want = ops.wtconv_gated_fwd(x, gate, up)
    x[1, 3] = float("nan")
    got = ops.wtconv_gated_fwd(x, gate, up)
    assert torch.isnan(got[1]).all()
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(got[keep], want[keep])


def test_small_and_large_values(ops):
    for size in (1e-18, 1e12):
        dh, x, gate, up = inputs(200, 96, 130, F32)
        x, gate = x * size, gate / size
        check_forward(ops.wtconv_gated_fwd(x, gate, up), x, gate, up, "silu")


def test_far_from_zero_and_masked_units(ops):
    for dtype in TYPES:
        dh, x, gate, up = inputs(150, 64, 96, dtype)
        gate[3] = -300 * x[0].sign()
        h = ops.wtconv_gated_fwd(x, gate, up, activation="silu")
        assert torch.isfinite(h).all() and float(h[0, 3].abs()) < 1e-6
        got = ops.wtconv_gated_bwd(dh, x, gate, up, activation="gelu")
        assert all(torch.isfinite(t).all() for t in got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_given_outputs_streams_and_graphs(ops, dtype):
    dh, x, gate, up = inputs(300, 90, 130, dtype)
    h, grads = ops.wtconv_gated_fwd(x, gate, up), ops.wtconv_gated_bwd(dh, x, gate, up)
    side = torch.cuda.Stream()
    outs = [torch.empty_like(t) for t in (h, *grads)]
    side.wait_stream(torch.cuda.current_stream())
    assert ops.wtconv_gated_fwd(x, gate, up, h=outs[0], stream=side) is outs[0]
    ops.wtconv_gated_bwd(dh, x, gate, up, dx=outs[1], dgate=outs[2], dup=outs[3], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (h, *grads)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ch, cg = ops.wtconv_gated_fwd(x, gate, up), ops.wtconv_gated_bwd(dh, x, gate, up)
    up.neg_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ch, -h) and torch.equal(cg[2], grads[2]) and torch.equal(cg[1], -grads[1])


def test_what_lies_behind_the_last_row_stays(ops):
    for dtype in TYPES:
        dh, x, gate, up = inputs(131, 40, 72, dtype)
        buf = torch.full((140, 72), 7.0, device="cuda", dtype=dtype)
        ops.wtconv_gated_fwd(x, gate, up, h=buf[:131])
        assert (buf[131:] == 7).all()
        bx, bw = torch.full((140, 40), 7.0, device="cuda", dtype=dtype), torch.full((2, 80, 40), 7.0, device="cuda", dtype=dtype)
        ops.wtconv_gated_bwd(dh, x, gate, up, dx=bx[:131], dgate=bw[0, :72], dup=bw[1, :72])
        assert (bx[131:] == 7).all() and (bw[:, 72:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_tensors_that_begin_anywhere(ops, dtype):
    for M, C, H in ((3, 24, 40), (140, 64, 96), (129, 33, 57)):
        dh0, x0, gate0, up0 = inputs(M, C, H, dtype)
        for offsets in ((1, 0, 0, 0), (0, 1, 3, 5), (3, 3, 3, 3), (8, 8, 8, 8)):
            def place(t, o):
                flat = torch.full((t.numel() + 40,), 7.0, device="cuda", dtype=dtype)
                flat[16 + o:16 + o + t.numel()] = t.flatten()
                return flat[16 + o:16 + o + t.numel()].view(t.shape), flat

            dh, x, gate, up = (place(t, o)[0] for t, o in zip((dh0, x0, gate0, up0), offsets))
            outs = [place(t * 0, o) for t, o in zip((dh0, x0, gate0, up0), offsets)]
            ops.wtconv_gated_fwd(x, gate, up, h=outs[0][0])
            check_forward(outs[0][0], x0, gate0, up0, "silu")
            ops.wtconv_gated_bwd(dh, x, gate, up, dx=outs[1][0], dgate=outs[2][0], dup=outs[3][0])
            check_backward(tuple(o[0] for o in outs[1:]), dh0, x0, gate0, up0, "silu", dtype)
            for t, flat in outs:
                at = t.storage_offset()
                assert (flat[:at] == 7).all() and (flat[at + t.numel():] == 7).all()


def test_refusals(ops):
    dh, x, gate, up = inputs(4, 32, 16, F32)
    q, s = ops.wtconv_quantize_rows(x)
    w, ws = ops.wtconv_quantize_rows(gate)
    for call in (lambda: ops.wtconv_gated_fwd(x.cpu(), gate, up), lambda: ops.wtconv_gated_fwd(x, gate, up[:8]),
                 lambda: ops.wtconv_gated_fwd(x, gate[:, :16], up[:, :16]), lambda: ops.wtconv_gated_fwd(x, gate.half(), up),
                 lambda: ops.wtconv_gated_fwd(x, gate, up, activation="relu"), lambda: ops.wtconv_gated_fwd(x.double(), gate, up),
                 lambda: ops.wtconv_gated_fwd(x, gate[:0], up[:0]), lambda: ops.wtconv_gated_fwd(x[:1].expand(4, 32), gate, up),
                 lambda: ops.wtconv_gated_fwd(x, gate, up, h=dh[:, :8]), lambda: ops.wtconv_gated_fwd(x, gate, up, h=dh.half()),
                 lambda: ops.wtconv_gated_fwd(gate, gate, up, h=gate), lambda: ops.wtconv_gated_bwd(dh[:3], x, gate, up),
                 lambda: ops.wtconv_gated_bwd(dh.half(), x, gate, up), lambda: ops.wtconv_gated_bwd(dh, x, gate, up, dgate=gate),
                 lambda: ops.wtconv_gated_bwd(dh, x, gate, up, dx=x), lambda: ops.wtconv_gated_q8(x, s, w, ws, w, ws),
                 lambda: ops.wtconv_gated_q8(q, s[:3], w, ws, w, ws), lambda: ops.wtconv_gated_q8(q, s, w, None, w, ws),
                 lambda: ops.wtconv_gated_q8(q[:, :8], s, w[:, :8], ws, w[:, :8], ws),
                 lambda: ops.wtconv_gated_q8(q, s, w, ws, w, ws, dtype=torch.float64)):
        with pytest.raises(ValueError):
            call()
    need = ops._gated_layout(x, gate, up, dh, "silu", ops.OP_GATED_BWD).ws
    with pytest.raises(wtconv.WtconvError):
        ops.wtconv_gated_bwd(dh, x, gate, up, workspace=torch.empty(max(need - 1, 0), dtype=torch.uint8, device="cuda"))
    buf = torch.zeros(4 * 32 + 8, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(wtconv.WtconvError):
        ops.wtconv_gated_q8(buf[8:].view(4, 32), s, w, ws, w, ws)
