"""The binding's checks of the block operators' arguments, on CPU tensors."""
import itertools

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import blockops


def stack(ts):
    """The binding's view of a list of matrices, without its check of the device."""
    s = blockops._Stack.__new__(blockops._Stack)
    s.tensors = list(ts)
    s.m, s.n = ts[0].shape
    s.ld = ts[0].stride(0)
    s.pointers = [t.data_ptr() for t in ts]
    return s


def elements(t):
    m, n = t.shape
    return {t.storage_offset() + i * t.stride(0) + j for i in range(m) for j in range(n)}


def refused(ts):
    try:
        stack(ts).separate("w")
    except ValueError:
        return True
    return False


def test_matrices_that_share_elements_with_one_further_on():
    # side by side with the second, which begins between the first and the third
    flat = torch.zeros(64)
    at = lambda o: flat[o:].as_strided((2, 4), (10, 1), o)  # noqa: E731
    ts = [at(0), at(4), at(10)]
    assert elements(ts[0]) & elements(ts[2])
    assert refused(ts)
    assert not refused([at(0), at(4), at(20)])


def test_overlap_of_lists_agrees_with_the_elements():
    flat = torch.zeros(400)
    for m, n, ld in ((2, 4, 10), (3, 3, 9), (1, 5, 12), (3, 4, 4), (4, 1, 3)):
        for offsets in itertools.combinations(range(0, 34, 2 if n > 2 else 1), 3):
            ts = [flat.as_strided((m, n), (ld, 1), o) for o in offsets]
            sets = [elements(t) for t in ts]
            share = any(a & b for a, b in itertools.combinations(sets, 2))
            assert refused(ts) == share, (m, n, ld, offsets)


def test_polynomials_beyond_the_range_have_no_workspace():
    from memory_bound_cnn_wtconv2d_gb300 import build
    import ctypes
    build.build()
    L = blockops.lib()
    size = lambda abc, steps: L.wtconv_ns_workspace_size(  # noqa: E731
        ctypes.byref(blockops.NsDesc(2, 300, 400, 0, steps, *abc, 1e-7)))
    for abc, steps in (((16.0, 0.0, 0.0), 1), ((2.0, 0.0, 0.0), 5), ((16.0, 16.0, 16.0), 1), (blockops.NS_COEFFICIENTS, 64),
                       ((1.5, -0.5, 0.0), 64), ((1.875, -1.25, 0.375), 64), ((2.0, -1.5, 0.5), 64), ((-1.0, 0.0, 0.0), 64)):
        assert size(abc, steps) > 0, (abc, steps)
    for abc, steps in (((2.0, 0.0, 0.0), 6), ((16.0, 16.0, 16.0), 2), ((1.1, 0.0, 0.0), 64), ((0.0, 0.0, 16.0), 3),
                       ((-16.0, 16.0, -16.0), 2)):
        assert size(abc, steps) == 0, (abc, steps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_a_resumed_optimiser_has_its_buffers_in_float32(dtype):
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    shapes = [(6, 4), (4, 6), (3, 5, 1, 1), (2, 2)]
    new = lambda: [torch.nn.Parameter(torch.randn(s).to(dtype)) for s in shapes]  # noqa: E731
    ps = new()
    opt = Muon([{"params": ps[:2]}, {"params": ps[2:], "lr": 0.5}], lr=0.1)
    for p in ps[:3]:  # the last has not had a gradient
        opt.state[p]["buffer"] = torch.randn(p.shape)
    saved = opt.state_dict()
    qs = new()
    again = Muon([{"params": qs[:2]}, {"params": qs[2:]}], lr=0.3)
    again.load_state_dict(saved)
    assert [g["lr"] for g in again.param_groups] == [0.1, 0.5]
    for p, q in zip(ps[:3], qs):
        b = again.state[q]["buffer"]
        assert b.dtype is torch.float32 and torch.equal(b, opt.state[p]["buffer"])
        assert b.data_ptr() != opt.state[p]["buffer"].data_ptr()
    assert not again.state[qs[3]]


def refuses(call):
    try:
        call()
    except ValueError:
        return True
    return False


def test_refusals_do_not_depend_on_earlier_calls(monkeypatch):
    from memory_bound_cnn_wtconv2d_gb300 import build
    build.build()
    monkeypatch.setattr(blockops._c, "_on_cuda", lambda t: True)
    x = torch.zeros(2, 3, 8)
    s = stack([torch.zeros(20, 30)])
    s.dtype, s.device = torch.float32, torch.device("cpu")
    layout = lambda groups: blockops._gn_layout(x, None, groups, 1e-5, "none")  # noqa: E731
    desc = lambda steps: blockops._ns_desc(s, 1, steps, blockops.NS_COEFFICIENTS, 1e-7)  # noqa: E731
    assert refuses(lambda: layout(4.0)) and refuses(lambda: desc(5.0))
    assert layout(4) is layout(4) and desc(5) is desc(5)
    assert refuses(lambda: layout(4.0)) and refuses(lambda: desc(5.0))


@pytest.mark.parametrize("decay", [0.0, 0.05])
def test_the_weight_decay_asked_for_is_that_of_every_parameter(decay):
    from memory_bound_cnn_wtconv2d_gb300.block import WTConvBlock, block_optimizers
    for opt in block_optimizers(WTConvBlock(16, num_groups=4), weight_decay=decay):
        assert [g["weight_decay"] for g in opt.param_groups] == [decay]
