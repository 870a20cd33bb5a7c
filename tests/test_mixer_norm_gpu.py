"""RMS norm with the residual's addition against a plain float64 implementation.

Tolerances, derived before any run.  A float32 value of y or dx comes from a
handful of float32 operations (2^-24 relative each) and a sum over the row
whose relative error stays below 2^-24 times the few dozen additions a lane and
its tree make: 1e-5 relative to the terms' root mean square is far above that.
(dx is rstd w dy less a sum; in a row of one channel the two cancel but for eps,
and the rounding that stays is that of rstd w dy, not of their difference.)  16-bit results: one
rounding to nearest more, eps / 2 relative at most.  dweight: a float32 sum in
blocks, relative to the root of the sum of squares of its terms 1e-5.  An 8-bit
value is off by half a step of e4m3 at most: 2^-4 relative, or 2^-10 (half of
the smallest step) absolute; next to a border the float32 value may fall on the
other side, which adds 1e-5 of the value.
"""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import mixerops
    return mixerops


def half(dtype):
    return 0.0 if dtype is F32 else torch.finfo(dtype).eps / 2


def near(got, want, dtype, slack=1e-5, terms=None):
    """One rounding of each value, and `slack` of the root mean square (of the
    terms that the values are differences of)."""
    assert got.shape == want.shape
    rms = (want if terms is None else terms).square().mean().sqrt()
    off = (got.double() - want).abs() - half(dtype) * want.abs() - slack * torch.maximum(rms, want.abs())
    if dtype is F16:
        off = off - 2.0 ** -25  # below the normal range
    assert got.dtype == dtype and (not want.numel() or float(off.max()) <= 0), float(off.max() / rms)


def inputs(M, C, dtype, seed=0, residual=True, weight=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(M, C) * torch.exp(0.5 * r(C))).to(dtype)
    return (x, r(M, C).to(dtype) if residual else None, 1 + 0.2 * r(C) if weight else None, r(M, C).to(dtype),
            r(M, C).to(dtype))


def forward64(x, r, w, eps):
    t = x.double() + (0 if r is None else r.double())
    rstd = (t.square().mean(-1) + eps).rsqrt()
    return t * rstd[..., None] * (1 if w is None else w.double()), t, rstd


def backward64(dy, t, rstd, w, dt):
    t, dy, rstd = t.double(), dy.double(), rstd.double()[..., None]
    xh, wd = t * rstd, dy * (1 if w is None else w.double())
    dx = rstd * (wd - xh * (wd * xh).mean(-1, keepdim=True)) + (0 if dt is None else dt.double())
    return dx, dy * xh, rstd * wd


SHAPES = [(1, 1), (1, 768), (3, 7), (49, 96), (130, 90), (1000, 33), (17, 257), (5, 1024), (2, 1030), (7, 2048), (3, 4100),
          (2, 8192), (2, 16384), (1, 16383), (20011, 64), (70000, 24), (513, 1000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C", SHAPES)
def test_forward_and_backward(ops, M, C, dtype):
    for residual, weight in ((True, True), (False, False)):
        x, r, w, dy, dt = inputs(M, C, dtype, M + C, residual, weight)
        y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=r)
        y64, t64, rstd64 = forward64(x, r, w, 1e-6)
        near(y, y64, dtype)
        near(total, t64, dtype, 1e-6)
        near(rstd, rstd64, F32)
        if r is None:
            assert total is x
        dt = dt if residual else None
        dx, dw = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt)
        dx64, terms, first = backward64(dy, total, rstd, w, dt)
        near(dx, dx64, dtype, terms=torch.maximum(first.abs(), dx64.abs()))
        size = terms.square().sum(0).sqrt()
        assert dw.dtype is F32 and float(((dw.double() - terms.sum(0)).abs() - 1e-5 * size).max()) <= 0
        again = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt)
        assert torch.equal(again[1], dw) and torch.equal(again[0], dx)
        only, none = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt, need_dweight=False)
        assert none is None and torch.equal(only, dx)


def in_8_bits(q, scale, y64):
    s64 = y64.abs().amax(-1) / 448
    near(scale, s64, F32)
    want = y64 / s64[..., None].clamp_min(2.0 ** -120)
    off = (q.double() - want).abs() - torch.maximum(want.abs() * (2.0 ** -4 + 1e-5), torch.full_like(want, 2.0 ** -10 + 1e-5))
    assert q.dtype is torch.float8_e4m3fn and float(off.max()) <= 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C", [s for s in SHAPES if s[1] > 1])
def test_8_bit_output(ops, M, C, dtype):
    for residual in (True, False):
        x, r, w, _, _ = inputs(M, C, dtype, M + C, residual)
        q, scale, total = ops.wtconv_rms_norm_q8(x, w, residual=r)
        y64, t64, _ = forward64(x, r, w, 1e-6)
        in_8_bits(q, scale, y64)
        near(total, t64, dtype, 1e-6)
    q, scale = ops.wtconv_quantize_rows(x)
    in_8_bits(q, scale, x.double())


@pytest.mark.parametrize("dtype", TYPES)
def test_slices_and_leading_axes(ops, dtype):
    wide = torch.randn(3, 5, 7, 200, device="cuda").to(dtype)
    for a, b in ((0, 96), (100, 196), (1, 64), (3, 200)):
        x, r, dy = wide[..., a:b], wide.flip(0)[..., a:b].contiguous(), wide.flip(1)[..., a:b]
        y, total, rstd = ops.wtconv_rms_norm_fwd(x, residual=r)
        y64, t64, rstd64 = forward64(x, r, None, 1e-6)
        near(y, y64, dtype)
        near(total, t64, dtype, 1e-6)
        assert y.is_contiguous() and rstd.shape == (3, 5, 7)
        q, scale, _ = ops.wtconv_rms_norm_q8(x, residual=r)
        in_8_bits(q, scale, y64)
        dx, dw = ops.wtconv_rms_norm_bwd(dy, x, rstd, dtotal=x)
        dx64 = backward64(dy, x, rstd, None, x)[0]
        near(dx, dx64, dtype)
    row = wide[0, 0, 0]
    near(ops.wtconv_rms_norm_fwd(row)[0], forward64(row, None, None, 1e-6)[0], dtype)


def at_offset(shape, offset, dtype, fill=None):
    """A contiguous tensor that begins `offset` elements behind a 16-byte boundary, and
    the buffer around it."""
    n = 1
    for v in shape:
        n *= v
    flat = torch.full((n + 64,), 7.0, device="cuda").to(dtype)
    t = flat[32 + offset:32 + offset + n].view(shape)
    if fill is not None:
        t.copy_(fill)
    return t, flat


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,C", [(1, 1), (2, 3), (9, 5), (40, 7), (100, 90), (33, 91), (300, 257), (3, 1001), (1000, 13), (7, 8), (64, 96)])
def test_rows_that_begin_anywhere(ops, M, C, dtype):
    x0, r0, w, dy0, dt0 = inputs(M, C, dtype, C)
    q8 = torch.float8_e4m3fn
    for offsets in ((0, 0, 0, 0), (1, 1, 1, 1), (3, 3, 3, 3), (0, 1, 2, 3), (5, 5, 5, 0), (7, 7, 7, 7)):
        x, r, dy, dt = (at_offset((M, C), o, dtype, v)[0] for o, v in zip(offsets, (x0, r0, dy0, dt0)))
        outs = [at_offset((M, C), o, t) for o, t in zip((offsets[0], offsets[1], offsets[0], offsets[3]), (dtype, dtype, q8, dtype))]
        y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=r, y=outs[0][0], total=outs[1][0])
        y64, t64, _ = forward64(x0, r0, w, 1e-6)
        near(y, y64, dtype)
        near(total, t64, dtype, 1e-6)
        q, scale, _ = ops.wtconv_rms_norm_q8(x, w, residual=r, q=outs[2][0])
        in_8_bits(q, scale, y64)
        dx, dw = ops.wtconv_rms_norm_bwd(dy, x, rstd, w, dtotal=dt, dx=outs[3][0])
        dx64, terms, first = backward64(dy0, x0, rstd, w, dt0)
        near(dx, dx64, dtype, terms=torch.maximum(first.abs(), dx64.abs()))
        assert float(((dw.double() - terms.sum(0)).abs() - 1e-5 * terms.square().sum(0).sqrt()).max()) <= 0
        for t, flat in outs:  # nothing around the outputs is touched
            at = t.storage_offset()
            around = torch.cat([flat[:at].float(), flat[at + M * C:].float()])
            assert (around == 7).all()


def test_rows_of_zeros_and_of_extremes(ops):
    x = torch.randn(9, 320, device="cuda")
    x[2] = 0
    x[4] *= 1e-18
    x[5] *= 1e17
    y, _, rstd = ops.wtconv_rms_norm_fwd(x, eps=0.0)
    keep = [i for i in range(9) if i != 2]
    near(y[keep], forward64(x[keep], None, None, 0.0)[0], F32)
    y, _, rstd = ops.wtconv_rms_norm_fwd(x, eps=1e-6)
    assert torch.equal(y[2], torch.zeros_like(y[2])) and float(rstd[2]) == pytest.approx(1e3, rel=1e-6)
    q, scale, _ = ops.wtconv_rms_norm_q8(x)
    assert not q[2].float().any() and 0 < float(scale[2]) <= 2.0 ** -120
    q, scale = ops.wtconv_quantize_rows(torch.cat([x, x * 0 + 3e38]))
    assert torch.isfinite(q.float()).all() and float(q[-1].float().min()) == 448


def test_infinities_and_nans_stay_in_their_row(ops):
    x = torch.randn(6, 130, device="cuda")
    want = ops.wtconv_rms_norm_fwd(x)[0]
    bad = x.clone()
    bad[1, 5], bad[3, 0] = float("inf"), float("nan")
    y = ops.wtconv_rms_norm_fwd(bad)[0]
    keep = [0, 2, 4, 5]
    assert torch.equal(y[keep], want[keep])
    assert torch.isnan(y[1, 5]) and torch.isnan(y[3]).all()
    for q, scale in (ops.wtconv_quantize_rows(bad), ops.wtconv_rms_norm_q8(bad)[:2]):
        assert not torch.isfinite(scale[[1, 3]]).any() and torch.isfinite(scale[keep]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_empty(ops, dtype):
    x = torch.empty(0, 5, 64, device="cuda", dtype=dtype)
    y, total, rstd = ops.wtconv_rms_norm_fwd(x, residual=x.clone())
    assert y.shape == total.shape == x.shape and rstd.shape == (0, 5)
    q, scale, _ = ops.wtconv_rms_norm_q8(x)
    assert q.shape == x.shape and scale.shape == (0, 5)
    dx, dw = ops.wtconv_rms_norm_bwd(x, x, rstd)
    assert dx.shape == x.shape and not dw.any() and dw.shape == (64,)


def test_given_outputs_and_streams(ops):
    x, r, w, dy, dt = inputs(300, 96, F16)
    y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=r)
    outs = [torch.empty_like(t) for t in (y, total, rstd)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.wtconv_rms_norm_fwd(x, w, residual=r, y=outs[0], total=outs[1], rstd=outs[2], stream=side)
    side.synchronize()
    assert all(a is b for a, b in zip(got, outs)) and all(torch.equal(a, b) for a, b in zip(got, (y, total, rstd)))
    dx, dw = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt)
    a, b = torch.empty_like(dx), torch.empty_like(dw)
    ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt, dx=a, dweight=b)
    assert torch.equal(a, dx) and torch.equal(b, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dt)
        f = ops.wtconv_rms_norm_fwd(x, w, residual=r)
    dy.neg_()
    x.neg_()
    r.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(f[0], -y) and torch.equal(f[2], rstd) and torch.equal(g[1], -dw)


def test_refusals(ops):
    x = torch.randn(4, 64, device="cuda")
    w, rstd = torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    for call in (lambda: ops.wtconv_rms_norm_fwd(x.cpu()), lambda: ops.wtconv_rms_norm_fwd(x.double()),
                 lambda: ops.wtconv_rms_norm_fwd(x.t()), lambda: ops.wtconv_rms_norm_fwd(x[:1].expand(4, 64)),
                 lambda: ops.wtconv_rms_norm_fwd(x, w[:63]), lambda: ops.wtconv_rms_norm_fwd(x, w.half()),
                 lambda: ops.wtconv_rms_norm_fwd(x, residual=x[:3]), lambda: ops.wtconv_rms_norm_fwd(x, residual=x.half()),
                 lambda: ops.wtconv_rms_norm_fwd(x, eps=-1.0), lambda: ops.wtconv_rms_norm_fwd(x, eps=float("nan")),
                 lambda: ops.wtconv_rms_norm_fwd(x, y=x), lambda: ops.wtconv_rms_norm_fwd(x, y=x.half()),
                 lambda: ops.wtconv_rms_norm_fwd(x, total=torch.empty_like(x)),
                 lambda: ops.wtconv_rms_norm_fwd(x, residual=w.expand(4, 64)),
                 lambda: ops.wtconv_rms_norm_bwd(x, x, None), lambda: ops.wtconv_rms_norm_bwd(x, x, rstd[:3]),
                 lambda: ops.wtconv_rms_norm_bwd(x.half(), x, rstd), lambda: ops.wtconv_rms_norm_bwd(x, x, rstd, dx=x),
                 lambda: ops.wtconv_rms_norm_q8(x, q=torch.empty_like(x)), lambda: ops.wtconv_quantize_rows(x[:, :0])):
        with pytest.raises(ValueError):
            call()
    from memory_bound_cnn_wtconv2d_gb300 import wtconv
    with pytest.raises(wtconv.WtconvError):
        ops.wtconv_rms_norm_fwd(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(wtconv.WtconvError):
        ops.wtconv_rms_norm_bwd(x, x, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
