"""What the clipping of a module's gradients refuses, without a GPU."""
import pytest
import torch

from memory_bound_cnn_wtconv2d_gb300.clip import clip_grad_norm_


def test_a_norm_type_is_not_taken_for_eps():
    # torch.nn.utils.clip_grad_norm_(parameters, max_norm, norm_type)
    p = torch.nn.Parameter(torch.ones(3))
    for more in ((2.0,), (2.0, True)):
        with pytest.raises(TypeError):
            clip_grad_norm_([p], 1.0, *more)
    assert float(clip_grad_norm_([p], 1.0, eps=0.0, error_if_nonfinite=True)) == 0  # no gradient


def test_gradients_that_are_refused():
    p = torch.nn.Parameter(torch.ones(3))
    p.grad = torch.ones(3)  # on the host
    with pytest.raises(ValueError, match="CUDA"):
        clip_grad_norm_(p, 1.0)
