"""The mixer's operators over many rows: norms of rows that no CTA holds, with more
rows than CTAs, and gradients of matrices that are sums over millions of rows."""
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
    yield mixerops
    torch.cuda.empty_cache()


# Every row of more channels than 256 lanes hold (32 values a lane forward, backward 24 of 16
# bits or 16 of float32; 8 where tensors are read value by value, which other offsets
# bring about), and with an odd width.
@pytest.mark.parametrize("dtype,C,offsets", [
    (F32, 4100, (0, 0, 0)), (F32, 5001, (0, 0, 0)), (F32, 8200, (0, 0, 0)), (F32, 2050, (0, 1, 0)),
    (F16, 6152, (0, 0, 0)), (F16, 9001, (0, 0, 0)), (F16, 2049, (0, 1, 3)),
    (BF16, 16384, (0, 0, 0)), (BF16, 8200, (0, 0, 1)), (BF16, 6200, (5, 5, 5))])
def test_rows_that_no_cta_holds(ops, dtype, C, offsets):
    from test_mixer_norm_gpu import at_offset, backward64, forward64, in_8_bits, inputs, near
    M = 2700  # three turns of the CTAs, and dw's ranges of rows hold three and fewer
    x, r, w, dy, dt = inputs(M, C, dtype, C)
    x, r, dy = (at_offset((M, C), o, dtype, v)[0] for o, v in zip(offsets, (x, r, dy)))
    y, total, rstd = ops.wtconv_rms_norm_fwd(x, w, residual=r)
    y64, t64, rstd64 = forward64(x, r, w, 1e-6)
    near(y, y64, dtype)
    near(total, t64, dtype, 1e-6)
    near(rstd, rstd64, F32)
    q, scale, total8 = ops.wtconv_rms_norm_q8(x, w, residual=r)
    in_8_bits(q, scale, y64)
    assert torch.equal(total8, total)
    in_8_bits(*ops.wtconv_quantize_rows(x), x.double())
    del y64, t64
    x.copy_(total)
    dx, dw = ops.wtconv_rms_norm_bwd(dy, x, rstd, w, dtotal=dt)
    dx64, terms, first = backward64(dy, x, rstd, w, dt)
    near(dx, dx64, dtype, terms=torch.maximum(first.abs(), dx64.abs()))
    size = terms.square().sum(0).sqrt()
    assert float(((dw.double() - terms.sum(0)).abs() - 1e-5 * size).max()) <= 0
    again = ops.wtconv_rms_norm_bwd(dy, x, rstd, w, dtotal=dt)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_gradients_that_are_sums_over_millions_of_rows(ops, dtype):
    """All terms of one sign, and every product and dg, du exact: what is off is the sums'.
    A sum leaves the tensor core after 256 k blocks of 64 rows at most: 1024 additions of
    sixteen products, which truncate, each by less than 2^-23 of a sum that grows to the
    result, so half of that on the way: 2^-14.  The splits, 1300 here at most, are added by
    float32 additions that round: 1300 * 2^-24 / 2 = 2^-14.7.  One rounding to the type
    follows.  2^-13 stands for the two."""
    M, C, H = 1 << 24, 16, 256
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = (torch.randint(8, 16, (M, C), generator=g, device="cuda", dtype=torch.int32) / 8).to(dtype)
    # hidden unit h sees channel h % 16 alone, and has an upstream gradient of its own
    gate = torch.eye(C, device="cuda").repeat(H // C, 1).to(dtype)
    size = (8 + torch.arange(H, device="cuda") // C % 8) * 2.0 ** -16
    dh = size.to(dtype).expand(M, H).contiguous()
    gram = torch.zeros(C, C, dtype=torch.float64, device="cuda")
    for part in x.split(1 << 20):
        gram += part.double().T @ part.double()
    want = size.double()[:, None] * gram.repeat(H // C, 1)
    _, dgate, dup = ops.wtconv_gated_bwd(dh, x, gate, gate, activation="none", need_dx=False)
    for got in (dgate, dup):
        off = (got.double() / want - 1).abs().max()
        assert float(off) <= torch.finfo(dtype).eps / 2 + 2.0 ** -13, float(off)
