"""A block's scales are numbers: one that autograd is asked to learn would get no gradient."""
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R


@pytest.mark.parametrize("name", ["scale", "residual_scale"])
def test_a_learned_scale_is_refused(name):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    learned = torch.tensor(0.7, requires_grad=True)
    with pytest.raises(TypeError, match=f"{name} .*gradient"):
        R.rmsnorm_block_train(x, x, w, **{name: learned})


def test_a_tensor_without_a_gradient_is_a_number():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    with pytest.raises(TypeError, match="CUDA"):   # the next check
        R.rmsnorm_block_train(x, x, w, scale=torch.tensor(0.7))
