"""A saved and resumed optimiser takes the same steps as one that went on."""
import io

import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300 import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_resumed_steps_are_the_same(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from memory_bound_cnn_wtconv2d_gb300.muon import Muon
    torch.manual_seed(0)
    ps = [torch.nn.Parameter((0.1 * torch.randn(s, device="cuda")).to(dtype)) for s in ((48, 20), (20, 48), (200, 130), (8, 8, 1, 1))]
    grads = [[(1e-3 * torch.randn(p.shape, device="cuda")).to(dtype) for p in ps] for _ in range(4)]

    def steps(opt, params, gs):
        for g in gs:
            for p, v in zip(params, g):
                p.grad = v.clone()
            opt.step()

    opt = Muon(ps, lr=0.05, weight_decay=0.1)
    steps(opt, ps, grads[:2])
    file = io.BytesIO()
    torch.save({"opt": opt.state_dict(), "params": [p.detach() for p in ps]}, file)
    steps(opt, ps, grads[2:])
    file.seek(0)
    loaded = torch.load(file, map_location="cpu")
    qs = [torch.nn.Parameter(p.cuda()) for p in loaded["params"]]
    again = Muon(qs, lr=1.0)
    again.load_state_dict(loaded["opt"])
    steps(again, qs, grads[2:])
    for p, q in zip(ps, qs):
        assert torch.equal(p, q)
        assert torch.equal(opt.state[p]["buffer"], again.state[q]["buffer"])
