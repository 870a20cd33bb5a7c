"""Group norm of more samples than the GPU holds CTAs of the streamed form at
once (two for each of its SMs), against float64, with the tolerances of the
other group norm tests."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build
from test_block_norm_gpu import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


# whole samples that no CTA holds, few rows of many channels, samples just above and far above the places
@pytest.mark.parametrize("shape,G,dtype,act", [((305, 41, 40, 24), 3, F32, "silu"), ((400, 40, 40, 48), 6, F16, "gelu"),
                                               ((1000, 7, 7, 300), 25, F32, "none"), ((700, 7, 7, 768), 32, BF16, "gelu"),
                                               ((3000, 5, 5, 260), 4, F16, "silu"), ((310, 90, 1100), 10, BF16, "none"), ((512, 7, 7, 768), 32, F32, "gelu"),
                                               ((400, 14, 14, 256), 32, F32, "silu")])
def test_more_samples_than_places(ops, shape, G, dtype, act):
    x, dy, w, b = inputs(shape, dtype, seed=shape[0])
    check_forward(ops, x, G, w, b, act)
    check_backward(ops, dy, x, G, w, b, act)
