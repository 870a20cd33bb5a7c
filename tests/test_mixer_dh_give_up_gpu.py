"""A wait for a copy of dh that gives up, without a GPU fault: the hook
wtconv_test_dh_timeout arms every warp's first barrier of dh with more bytes than
its copy delivers.  What is made of a dh that did not come is NaN, and the next call
is right."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import mixerops
    return mixerops


# one tile a CTA, one and two stretches a warp, several tiles, pairs, ragged ends
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,C,H", [(60, 64, 96), (300, 200, 520), (129, 40, 48), (5000, 96, 304), (30000, 40, 104)])
def test_gradients_of_a_dh_that_did_not_come_are_nan(ops, M, C, H, dtype):
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    r = lambda *s: torch.randn(*s, device="cuda").to(dtype)  # noqa: E731
    dh, x, gate, up = r(M, H), r(M, C), r(H, C), r(H, C)
    grads = ops.wtconv_gated_bwd(dh, x, gate, up)
    assert blockops.wtconv_block_device_faults() == 0
    outs = [torch.zeros_like(t) for t in grads]
    ops.wtconv_test_dh_timeout(True)
    try:
        ops.wtconv_gated_bwd(dh, x, gate, up, dx=outs[0], dgate=outs[1], dup=outs[2])
        torch.cuda.synchronize()
    finally:
        ops.wtconv_test_dh_timeout(False)
    # every row of dx and every hidden unit's gradient has a value of dg or du that was held up
    assert all(torch.isnan(t).all() for t in outs) and blockops.wtconv_block_device_faults() > 0
    assert all(torch.equal(a, b) for a, b in zip(ops.wtconv_gated_bwd(dh, x, gate, up), grads))
    assert blockops.wtconv_block_device_faults() == 0
