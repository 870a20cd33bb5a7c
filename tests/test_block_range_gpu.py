"""Newton-Schulz away from the usual sizes: polynomials that make the matrix
grow or shrink, gradients far below eps, very long rows.  Against float64.

Tolerances, derived before any run: as in the tests of the usual sizes, 1e-5
relative 2-norm for float32 (operands of 22 bits, float32 sums) and 5e-3 for
16-bit types (operands of 11 bits).  The polynomials here have terms of one
sign, so that none of what the terms carry is lost in their sum, and at most
five steps whose relative slope is at most 5.
"""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build, wtconv

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TOL = {F32: 1e-5, F16: 5e-3, BF16: 5e-3}
ABC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


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
    return float((a.double() - b).norm() / b.norm())


def random(*shape, dtype=F32, seed=0, size=1e-3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dtype)


def one_entry(m, n, dtype):
    g = torch.zeros(m, n, device="cuda", dtype=dtype)
    g[m // 2, n // 3] = -0.25
    return g


GROWING = [((16.0, 0.0, 0.0), 1), ((2.0, 0.0, 0.0), 5), ((4.0, 1.0, 0.5), 1), ((1.5, 0.5, 0.25), 2), ((16.0, 16.0, 16.0), 1)]


@pytest.mark.parametrize("abc,steps", GROWING)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n", [(90, 700), (4, 6), (600, 1100), (1300, 1100)])
def test_growing_polynomials(ops, m, n, dtype, abc, steps):
    for g in (random(m, n, dtype=dtype, seed=m), one_entry(m, n, dtype)):
        assert rel(ops.wtconv_orthogonalize(g, steps=steps, coefficients=abc), ns64(g, steps, abc)) <= TOL[dtype]


def test_one_entry_of_a_large_matrix(ops):
    g = one_entry(4096, 4096, F32)
    assert rel(ops.wtconv_orthogonalize(g, steps=1, coefficients=(16.0, 0.0, 0.0)), ns64(g, 1, (16.0, 0.0, 0.0))) <= 1e-5


def test_polynomials_that_leave_the_range_are_refused(ops):
    g = random(70, 90)
    out = torch.full_like(g, 7.0)
    for abc, steps in (((2.0, 0.0, 0.0), 20), ((16.0, 16.0, 16.0), 2), ((1.1, 0.0, 0.0), 64)):
        with pytest.raises(wtconv.WtconvError) as e:
            ops.wtconv_orthogonalize(g, steps=steps, coefficients=abc, out=out)
        assert e.value.status == wtconv.WTCONV_ERR_UNSUPPORTED
    assert float((out - 7).abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", [(300, 700), (700, 90), (5, 9), (1030, 640)])
@pytest.mark.parametrize("norm", [3e-8, 1e-10, 1e-12, 1e-15, 1e-17])
def test_norms_far_below_eps(ops, norm, m, n, dtype):
    # X = g / (|g| + eps) is tiny, and so is the result; its bits are asked for all the same
    g = random(2, m, n, seed=n, size=1.0)
    g[1] *= 1e6  # beside a matrix further up
    g = (g * (norm / float(g[0].norm()))).to(dtype)
    out = ops.wtconv_orthogonalize(g)
    for i in range(2):
        assert rel(out[i], ns64(g[i])) <= TOL[dtype]


@pytest.mark.parametrize("m,n", [(100, 300), (420, 300)])
def test_a_tiny_matrix_grows_to_an_orthogonal_one(ops, m, n):
    # 64 cubic steps from a norm of 1e-10 / 1e-7: 17 to come to 1, the rest converges.
    # Each rounds by 2^-22 of the result at most: 64 of them stay below 2e-5.
    g = random(m, n, seed=3, size=1.0)
    g *= 1e-10 / float(g.norm())
    out = ops.wtconv_orthogonalize(g, steps=64, coefficients=(1.5, -0.5, 0.0))
    want = ns64(g, 64, (1.5, -0.5, 0.0))
    assert abs(float(want.norm()) - min(m, n) ** 0.5) < 1e-6
    assert rel(out, want) <= 2e-5


@pytest.mark.parametrize("abc,steps", [((0.5, 0.0, 0.0), 20), ((0.25, 0.1, 0.0), 15), ((-0.75, 0.0, -0.1), 9)])
@pytest.mark.parametrize("m,n", [(90, 700), (600, 500)])
def test_shrinking_polynomials(ops, m, n, abc, steps):
    g = random(m, n, seed=5)
    # 20 roundings of 2^-22 at most
    assert rel(ops.wtconv_orthogonalize(g, steps=steps, coefficients=abc), ns64(g, steps, abc)) <= 1e-5


@pytest.mark.parametrize("m,n", [(60, 90), (300, 200)])
def test_optimizer_step_on_a_tiny_gradient(ops, m, n):
    w, g, b = torch.zeros(m, n, device="cuda"), random(m, n, seed=6, size=1e-14), torch.zeros(m, n, device="cuda")
    m64 = 0.05 * g.double()
    ops.wtconv_muon_step(w, g, b, lr=1.0, momentum=0.95, nesterov=False)
    assert rel(w, -ns64(m64)) <= 1e-5


@pytest.mark.parametrize("m,n", [(150, 4000), (4000, 150), (140, 12000), (130, 32768), (32768, 130), (700, 9000)])
def test_very_long_rows(ops, m, n):
    # the diagonal of X X^T is a sum of n squares
    g = random(m, n, seed=m)
    assert rel(ops.wtconv_orthogonalize(g), ns64(g)) <= 1e-5
    # an orthogonal matrix stays one: every step starts from the largest sums there are
    q = ops.wtconv_orthogonalize(g, steps=20, coefficients=(1.5, -0.5, 0.0))
    assert rel(q, ns64(g, 20, (1.5, -0.5, 0.0))) <= 1e-5


def step64(w, g, b, lr, mu, wd, scale):
    b = mu * b.double() + (1 - mu) * g.double()
    return (1 - lr * wd) * w.double() - lr * scale * ns64(mu * b + (1 - mu) * g.double()), b


@pytest.mark.parametrize("count,m,n", [(2, 1024, 2048), (1, 2048, 1024), (1, 300, 9000), (1, 9000, 300), (1, 1500, 1500),
                                       (3, 520, 1601)])
def test_optimizer_step_of_large_float32_matrices(ops, count, m, n):
    # weights of 0: what comes out is the direction, to the bits of a float32 stack
    w = torch.zeros(count, m, n, device="cuda")
    g, b = random(count, m, n, seed=n), random(count, m, n, seed=n + 1)
    want = [step64(w[i], g[i], b[i], 0.5, 0.9, 0.1, 1.5) for i in range(count)]
    ops.wtconv_muon_step(w, g, b, lr=0.5, momentum=0.9, weight_decay=0.1, scale=1.5)
    for i in range(count):
        assert rel(w[i], want[i][0]) <= 1e-5 and rel(b[i], want[i][1]) <= 1e-6
