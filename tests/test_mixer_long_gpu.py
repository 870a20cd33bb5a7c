"""The mixer's operators where offsets pass 2^31 elements: the rows at both ends and
around that border, against the same rows alone (which other tests hold against
float64), or where sums run over all rows, against sums over the few that are not
zero."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import mixerops
    yield mixerops
    torch.cuda.empty_cache()


def some_rows(M, C):
    """Slices of eight rows."""
    border = 2 ** 31 // C
    return [slice(0, 8), slice(border - 4, border + 4), slice(M - 8, M)]


def filled(M, C, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.zeros(M, C, dtype=dtype, device="cuda")
    for s in some_rows(M, C):
        t[s] = torch.randn(8, C, generator=g, device="cuda").to(dtype)
    return t


@pytest.mark.parametrize("C", [1024, 1001])
def test_norm(ops, C):
    M = 2 ** 31 // C + 99
    x, dy = filled(M, C, BF16, 0), filled(M, C, BF16, 1)
    w = torch.rand(C, device="cuda") + 0.5
    y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=x)
    rows = some_rows(M, C)
    for s in rows:
        want = ops.wtconv_rms_norm_fwd(x[s].clone(), w, residual=x[s].clone())
        # eight rows may be spread over other lanes: sums in another order
        assert torch.equal(total[s], want[1])
        torch.testing.assert_close(rstd[s], want[2], rtol=1e-6, atol=0)
        torch.testing.assert_close(y[s], want[0], rtol=2.0 ** -7, atol=0)
    assert not y[rows[0].stop:rows[1].start].any() and not total[rows[1].stop:rows[2].start].any()
    del y
    dx, dw = ops.wtconv_rms_norm_bwd(dy, total, rstd, w, dtotal=dy)
    xhat = torch.cat([total[s].double() * rstd[s].double()[:, None] for s in rows])
    want = (xhat * torch.cat([dy[s].double() for s in rows])).sum(0)
    assert float((dw.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())
    for s in rows:
        some, _ = ops.wtconv_rms_norm_bwd(dy[s].clone(), total[s].clone(), rstd[s].clone(), w, dtotal=dy[s].clone())
        # a value that the two orders leave on two sides of a border, next to terms of its size or above
        torch.testing.assert_close(dx[s], some, rtol=2.0 ** -7, atol=1e-5)
    del dx
    q, scale, _ = ops.wtconv_rms_norm_q8(total, w)
    for s in rows:
        want, sw, _ = ops.wtconv_rms_norm_q8(total[s].clone(), w)
        torch.testing.assert_close(scale[s], sw, rtol=1e-6, atol=0)
        # next steps of e4m3 at most
        torch.testing.assert_close(q[s].float(), want.float(), rtol=2.0 ** -3, atol=2.0 ** -9)


def test_norm_of_rows_far_apart(ops):
    M, C, stride = 20, 96, (1 << 27) + 8
    buf = torch.zeros((M - 1) * stride + C, dtype=F16, device="cuda")
    x = buf.as_strided((M, C), (stride, 1))
    x.copy_(torch.randn(M, C, device="cuda"))
    got, want = ops.wtconv_rms_norm_fwd(x), ops.wtconv_rms_norm_fwd(x.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    a, b = ops.wtconv_rms_norm_bwd(x, x, got[2], dtotal=x), ops.wtconv_rms_norm_bwd(x.contiguous(), x.contiguous(), got[2], dtotal=x.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("H", [264, 259])
def test_gated(ops, H):
    C, M = 16, 2 ** 31 // H + 777
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    gate, up = (torch.randn(H, C, generator=g, device="cuda").to(BF16) for _ in range(2))
    dh = filled(M, H, BF16, 3)
    rows = some_rows(M, H)
    x = torch.randn(M, C, generator=g, device="cuda").to(BF16)
    h = ops.wtconv_gated_fwd(x, gate, up)
    pick = lambda t: torch.cat([t[s] for s in rows])  # noqa: E731
    a, b = pick(x).double() @ gate.double().T, pick(x).double() @ up.double().T
    want = torch.nn.functional.silu(a) * b
    # products of 16 terms are good to 1e-6 of their size, of which the activation and the product make 3
    off = (pick(h).double() - want).abs() - 2.0 ** -8 * want.abs()
    assert float(off.max()) <= 3e-6 * float(a.abs().max() * b.abs().max())
    del h
    dx, dgate, dup = ops.wtconv_gated_bwd(dh, x, gate, up)
    few = ops.wtconv_gated_bwd(pick(dh), pick(x), gate, up)
    # the same sums but for their order (and zeros): a rounding to another side at most, after
    # float32 sums of 24 rows
    torch.testing.assert_close(pick(dx), few[0], rtol=2.0 ** -7, atol=1e-4)
    assert not dx[rows[0].stop:rows[1].start].any() and not dx[rows[1].stop:rows[2].start].any()
    torch.testing.assert_close(dgate, few[1], rtol=2.0 ** -7, atol=1e-4)
    torch.testing.assert_close(dup, few[2], rtol=2.0 ** -7, atol=1e-4)


def test_norm_of_a_long_list_and_clipping(ops):
    n = 2 ** 31 + 12345
    t = torch.full((n,), 2.0 ** -6, dtype=BF16, device="cuda")
    want = n ** 0.5 * 2.0 ** -6
    assert float(ops.wtconv_grad_norm([t])) == pytest.approx(want, rel=1e-6)
    ops.wtconv_clip_grads([t], 0.5 * want, eps=0.0)
    # a half of it, up to a float32 factor's rounding: within a step of bfloat16
    assert float(t.max()) <= 2.0 ** -7 * (1 + 2.0 ** -7) and float(t.min()) >= 2.0 ** -7 * (1 - 2.0 ** -7)


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16])
@pytest.mark.parametrize("M,C,H", [(9, 65536, 40), (300, 65536, 40), (9, 40, 65536), (300, 40, 65536), (1, 65536, 3), (1, 3, 65536)])
def test_the_widest_gated(ops, M, C, H, dtype):
    """A tensor core's addition of sixteen products is off by a step of float32 at most
    (it truncates), 2^-23 of a sum that stays below |x||w|: C / 16 of them; float32
    operands are added up in pieces of 512 values, six times 32 such additions and 128
    roundings, of which a deviate's root stays below 1e-5."""
    from test_mixer_gated_gpu import inputs, act64, grad64, half
    dh, x, gate, up = inputs(M, C, H, dtype)
    each = 1e-5 if dtype is torch.float32 else 1e-5 + C / 16 * 2.0 ** -23
    h = ops.wtconv_gated_fwd(x, gate, up)
    d = [t.double() for t in (dh, x, gate, up)]
    g, u = d[1] @ d[2].T, d[1] @ d[3].T
    a = act64(g, "silu")
    n = d[1].norm(dim=-1, keepdim=True) * each
    eg, eu = n * d[2].norm(dim=1), n * d[3].norm(dim=1)
    off = (h.double() - a * u).abs() - half(dtype) * 1.01 * (a * u).abs() - 1.2 * (eg * (u.abs() + eu) + eu * g.abs())
    assert float((off - (2.0 ** -25 if dtype is F16 else 0)).max()) <= 0
    dx, dgate, dup = ops.wtconv_gated_bwd(dh, x, gate, up)
    pg, pu = d[0] * u * grad64(g, "silu"), d[0] * a
    # dg and du: a rounding each and what g and u are off by; then sums over H (or M)
    rounding = 0 if dtype is torch.float32 else half(dtype)
    fg = rounding * pg.abs() + d[0].abs() * 1.2 * (eu + (u.abs() + eu) * eg)
    fu = rounding * pu.abs() + d[0].abs() * 1.2 * eg
    root = lambda p, q: ((p * p) @ (q * q)).sqrt()  # noqa: E731
    long = 1e-5 if dtype is torch.float32 else 1e-5 + 2 * H / 16 * 2.0 ** -23
    for got, want, size in ((dx, pg @ d[2] + pu @ d[3], 6 * (root(fg, d[2]) + root(fu, d[3])) + long * (root(pg, d[2]) + root(pu, d[3]))),
                            (dgate, pg.T @ d[1], 6 * root(fg.T, d[1]) + 1e-5 * root(pg.T, d[1])),
                            (dup, pu.T @ d[1], 6 * root(fu.T, d[1]) + 1e-5 * root(pu.T, d[1]))):
        off = (got.double() - want).abs() - half(dtype) * 1.01 * want.abs() - size - (2.0 ** -25 if dtype is F16 else 0)
        assert float(off.max()) <= 0, float(off.max())


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16])
def test_matrices_that_share_memory(ops, dtype):
    """One matrix twice, and two whose rows take turns: inputs may overlap."""
    from test_mixer_gated_gpu import check_backward, check_forward
    w, x, dh = (torch.randn(*s, device="cuda").to(dtype) for s in ((160, 72), (200, 72), (200, 80)))
    for gate, up in ((w[:80], w[:80]), (w[0::2], w[1::2]), (w[:80], w[80:]), (w[80:], w[1:81])):
        for rows in (3, 200):
            check_forward(ops.wtconv_gated_fwd(x[:rows], gate, up), x[:rows], gate, up, "silu")
        check_backward(ops.wtconv_gated_bwd(dh, x, gate, up), dh, x, gate, up, "silu", dtype)


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16])
@pytest.mark.parametrize("M,C,H", [(257, 16, 32768), (300, 40, 65536), (140, 40, 50000), (300, 32768, 16), (140, 50000, 40), (100, 20000, 300)])
def test_tiles_whose_warps_have_no_rows(ops, M, C, H, dtype):
    """A CTA takes tiles that end inside of the rows after whole ones, and short sums
    leave their warps little time: what a whole tile stored must have left its place.
    Against the same products of more rows, whose sums are the same or in another
    order: a step of the type at most; and from run to run, bit by bit."""
    from test_mixer_gated_gpu import inputs
    dh, x, gate, up = inputs(512, C, H, dtype)
    dh[M:] = 0
    whole = ops.wtconv_gated_fwd(x, gate, up)[:M]
    for _ in range(5):
        h = ops.wtconv_gated_fwd(x[:M], gate, up)
        assert float((h.double() - whole.double()).abs().max()) <= 2.0 ** -7 * float(whole.double().abs().max())
    first = ops.wtconv_gated_bwd(dh[:M], x[:M], gate, up)
    whole = ops.wtconv_gated_bwd(dh, x, gate, up)
    for _ in range(5):
        got = ops.wtconv_gated_bwd(dh[:M], x[:M], gate, up)
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        for a, b in zip(got, (whole[0][:M], *whole[1:])):
            assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -7 * float(b.double().abs().max())
