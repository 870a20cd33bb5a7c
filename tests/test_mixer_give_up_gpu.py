"""The give-up path of the gated kernels' bounded waits, without a GPU fault.

The hook wtconv_test_copy_timeout arms the first barrier of every product with
more bytes than its copies deliver, so that its wait runs out after about a
millisecond: the call has to return with the device usable, hand out NaN in the
place of what was held up, count the fault, and leave nothing behind that the
next call trips over.
"""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build, wtconv

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def faults():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops.wtconv_block_device_faults


def held(call):
    wtconv.wtconv_test_copy_timeout(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        wtconv.wtconv_test_copy_timeout(False)


# one tile a CTA, several, products with k shared out, and the three types
CASES = [(60, 64, 96, BF16), (5000, 96, 300, BF16), (30000, 40, 100, F16), (300, 200, 520, F32)]


@pytest.mark.parametrize("M,C,H,dtype", CASES)
def test_outputs_are_nan_and_the_next_call_is_right(faults, M, C, H, dtype):
    from memory_bound_cnn_wtconv2d_gb300 import mixerops as ops
    r = lambda *s: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    dh, x, gate, up = r(M, H), r(M, C), r(H, C), r(H, C)
    h, grads = ops.wtconv_gated_fwd(x, gate, up), ops.wtconv_gated_bwd(dh, x, gate, up)
    assert faults() == 0
    out = torch.zeros_like(h)
    held(lambda: ops.wtconv_gated_fwd(x, gate, up, h=out))
    assert torch.isnan(out).all() and faults() > 0
    outs = [torch.zeros_like(t) for t in grads]
    held(lambda: ops.wtconv_gated_bwd(dh, x, gate, up, dx=outs[0], dgate=outs[1], dup=outs[2]))
    assert all(torch.isnan(t).all() for t in outs) and faults() > 0
    assert torch.equal(ops.wtconv_gated_fwd(x, gate, up), h)
    assert all(torch.equal(a, b) for a, b in zip(ops.wtconv_gated_bwd(dh, x, gate, up), grads))
    assert faults() == 0


def test_8_bit_operands(faults):
    from memory_bound_cnn_wtconv2d_gb300 import mixerops as ops
    q = [t for m, n in ((500, 96), (200, 96), (200, 96)) for t in ops.wtconv_quantize_rows(torch.randn(m, n, device="cuda"))]
    h = ops.wtconv_gated_q8(*q)
    out = torch.zeros_like(h)
    held(lambda: ops.wtconv_gated_q8(*q, h=out))
    assert torch.isnan(out).all() and faults() > 0
    assert torch.equal(ops.wtconv_gated_q8(*q), h) and faults() == 0
