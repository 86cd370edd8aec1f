"""Group norm on the GPU where a value in the wrong place costs precision, or where one CTA or
cluster goes on to another sample: against the FP64 oracle, with the tolerances of
test_groupnorm_gpu.py where no other is derived here."""
from __future__ import annotations

import math

import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from test_groupnorm_gpu import DEV, randn

pytestmark = pytest.mark.gpu


def test_fp32_gelu_keeps_its_tail():
    # w = 0: z is b, one value a channel; with dy = 1 and one place db is the slope
    c, groups = 4096, 64
    z = torch.linspace(-12.5, 6, c, device=DEV)
    x, w = randn(1, 1, 1, c), torch.zeros(c, device=DEV)
    y, mean, rstd = R.groupnorm_fwd(x, w, z, groups, act="gelu")
    z64 = z.double()
    cdf = 0.5 * torch.erfc(-z64 / math.sqrt(2))
    phi = torch.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    # the normal distribution within 2^-20.5 of itself, one fma
    assert ((y[0, 0].double() - z64 * cdf).abs() <= 2.0 ** -20 * (z64 * cdf).abs()).all()
    dx, dw, db = R.groupnorm_bwd(torch.ones_like(x), x, mean, rstd, w, z, groups, "gelu")
    # exp2 2^-22, three FP32 roundings in z phi; the distribution as above; the sum's rounding
    e = (2.0 ** -21 * z64.abs() * phi + 2.0 ** -20 * cdf
         + 2.0 ** -23 * (cdf + z64 * phi).abs())
    assert ((db.double() - (cdf + z64 * phi)).abs() <= e).all()
