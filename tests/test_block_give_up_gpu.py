"""The give-up path of the matrix kernels' bounded waits, without a GPU fault.

The hook wtconv_test_copy_timeout makes one wait of every call run out after
about a millisecond (a barrier armed with more bytes than its copies deliver,
or products that are not committed): the call has to return with the device
usable, hand out no result, count the fault, and leave nothing behind that
the next call trips over.
"""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build, wtconv

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300 import blockops
    return blockops


def held(call):
    wtconv.wtconv_test_copy_timeout(True)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        wtconv.wtconv_test_copy_timeout(False)


# short matrices (a cluster each: one CTA, several), and the form of one launch
# over the GPU (wide, tall, more tiles than SMs)
CASES = [(2, 48, 60, F32), (3, 384, 96, BF16), (1, 128, 1024, F32), (2, 300, 200, BF16), (2, 333, 601, F32),
         (3, 1536, 384, F16)]


@pytest.mark.parametrize("count,m,n,dtype", CASES)
def test_orthogonalize_hands_out_nan(ops, count, m, n, dtype):
    g = torch.randn(count, m, n, device="cuda").to(dtype)
    want = ops.wtconv_orthogonalize(g)
    assert ops.wtconv_block_device_faults() == 0
    out = torch.zeros_like(g)
    held(lambda: ops.wtconv_orthogonalize(g, out=out))
    assert torch.isnan(out).all()
    assert ops.wtconv_block_device_faults() > 0
    assert torch.equal(ops.wtconv_orthogonalize(g), want)
    assert ops.wtconv_block_device_faults() == 0


@pytest.mark.parametrize("count,m,n,dtype", [CASES[1], CASES[2], CASES[4]])
def test_a_step_leaves_the_weights(ops, count, m, n, dtype):
    w, g = torch.randn(count, m, n, device="cuda").to(dtype), torch.randn(count, m, n, device="cuda").to(dtype)
    b = torch.zeros(count, m, n, device="cuda")
    before, good, gb = w.clone(), w.clone(), b.clone()
    held(lambda: ops.wtconv_muon_step(w, g, b, lr=0.1))
    assert torch.equal(w, before)
    assert ops.wtconv_block_device_faults() > 0
    ops.wtconv_muon_step(good, g, gb, lr=0.1)
    assert not torch.equal(good, before) and torch.isfinite(good).all()
    assert ops.wtconv_block_device_faults() == 0


@pytest.mark.parametrize("m,n", [(40, 60), (300, 200)])
def test_the_optimiser_says_so_at_a_later_step(ops, m, n):
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    p = torch.nn.Parameter(torch.randn(m, n, device="cuda"))
    opt = Muon([p], lr=0.1)
    p.grad = torch.randn(m, n, device="cuda")
    for first in (True, False):  # the first step's faults count too
        before = p.detach().clone()
        held(opt.step)
        assert torch.equal(p, before)
        with pytest.raises(RuntimeError, match="gave up"):
            opt.step()
        assert torch.equal(p, before)
        opt.step()
        opt.step()
        assert not torch.equal(p, before)
        if first:
            assert ops.wtconv_block_device_faults() > 0  # a reset between steps is no fault
            opt.step()
            opt.step()
    assert ops.wtconv_block_device_faults() > 0


def test_an_optimiser_does_not_answer_for_earlier_faults(ops):
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    g = torch.randn(2, 48, 60, device="cuda")
    held(lambda: ops.wtconv_orthogonalize(g))
    p = torch.nn.Parameter(torch.randn(40, 60, device="cuda"))
    opt = Muon([p], lr=0.1)
    p.grad = torch.randn(40, 60, device="cuda")
    for _ in range(3):
        opt.step()
        torch.cuda.synchronize()
    assert ops.wtconv_block_device_faults() > 0


def test_the_count_in_a_captured_step(ops):
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    p = torch.nn.Parameter(torch.randn(40, 60, device="cuda"))
    opt = Muon([p], lr=0.1)
    p.grad = torch.randn(40, 60, device="cuda")
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    before = p.detach().clone()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(p, before)
    opt.step()
    with pytest.raises(ValueError):
        ops.wtconv_block_device_faults_async(torch.zeros(1, dtype=torch.int32), "cuda")
    assert ops.wtconv_block_device_faults() == 0
