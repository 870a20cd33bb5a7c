"""Tiles of the gated product whose warps have no rows, value by value."""
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


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,C,H", [(257, 16, 32768), (300, 40, 65536), (140, 40, 50000), (300, 32768, 16), (140, 50000, 40), (100, 20000, 300)])
def test_every_value_of_tiles_that_end_behind_the_last_row(ops, M, C, H, dtype):
    """Each against float64 by one rounding of its own size and what its own sums leave
    (the bounds of the widest shapes), and from run to run the same bits."""
    from test_mixer_gated_gpu import inputs
    from test_mixer_long_gpu import test_the_widest_gated as by_value
    by_value(ops, M, C, H, dtype)
    dh, x, gate, up = inputs(M, C, H, dtype)
    h, grads = ops.wtconv_gated_fwd(x, gate, up), ops.wtconv_gated_bwd(dh, x, gate, up)
    for _ in range(5):
        assert torch.equal(ops.wtconv_gated_fwd(x, gate, up), h)
        assert all(torch.equal(a, b) for a, b in zip(ops.wtconv_gated_bwd(dh, x, gate, up), grads))
