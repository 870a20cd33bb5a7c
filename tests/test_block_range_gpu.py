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
