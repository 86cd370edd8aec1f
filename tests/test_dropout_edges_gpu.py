"""Dropout and the dropout RMSNorm on the GPU where their other tests do not look: the last elements
of a tensor, ring stages filled again, allocations through torch's dispatcher."""
from __future__ import annotations

import pytest
import torch

import rmsnorm_fwd_02_gb300 as R

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_kept_zeros_keep_their_sign(dtype, p):
    n = 2043                                      # whole vectors and the last three elements
    x = torch.full((n,), -0.0, dtype=dtype, device=DEV)
    kept = R.dropout_fwd(torch.ones_like(x), p, 3) != 0
    for y in (R.dropout_fwd(x, p, 3), R.dropout_bwd(x, p, 3)):
        assert not y.any() and torch.equal(y.signbit(), kept)
    ones = torch.ones(n, dtype=dtype, device=DEV)
    assert torch.equal(R.dropout_fwd(x, p, 3, residual=ones), ones)
