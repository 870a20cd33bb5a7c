"""Channels that a bias of the lowest finite value, or one far out, switches
off: silu and gelu are 0 there, and so are the gradients.  Against float64, with
the tolerances of the other group norm tests."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build
from test_block_norm_gpu import check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", [(2, 7, 9, 24), (3, 120, 130, 24)])
@pytest.mark.parametrize("bias", [LOWEST, -1e30, -1e20, -1e6])
def test_masked_channels(ops, shape, dtype, act, bias):
    x, dy, w, b = inputs(shape, dtype, seed=1)
    off = torch.zeros(24, dtype=torch.bool, device="cuda")
    off[[1, 4, 5, 23]] = True  # beside channels that stay, in one pair and apart
    masked = torch.where(off, bias, b)
    y, _, _ = check_forward(ops, x, 6, w, masked, act)
    assert float(y[..., off].abs().max()) <= 1e-15
    dx, dw, db = check_backward(ops, dy, x, 6, w, masked, act)
    assert float(dw[off].abs().max()) <= 1e-9 and float(db[off].abs().max()) <= 1e-9
