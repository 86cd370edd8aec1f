"""Dropout and the dropout RMSNorm on the GPU where their other tests do not look: the last elements
of a tensor, ring stages filled again, allocations through torch's dispatcher."""
from __future__ import annotations

import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import dropout as D

pytestmark = pytest.mark.gpu

DEV = "cuda"


def randn(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def half_step(v):
    """Half a bf16 step at the values v (float64)."""
    return 2.0 ** (v.abs().clamp(min=2.0 ** -126).log2().floor() - 8)


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


# sub-warp groups, narrow rows, 2 to 6 vectors a thread, the tensor-memory and the wide builds
@pytest.mark.parametrize("T,H", [(950000, 64), (240000, 264), (80000, 768), (40000, 1536),
                                 (30000, 2048), (16384, 4096), (12000, 6144), (9000, 8192)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_rings_that_go_round(T, H, with_dh):
    p, seed, offset = 0.2, 1 << 40, 77
    for op in (N.PLAN_FWD_RESIDUAL, N.PLAN_BWD_DH if with_dh else N.PLAN_BWD):
        plan = N.rmsnorm_train_launch_plan(H, op)
        ctas = 152 * min(2048 // plan["threads"], 228 * 1024 // (plan["smem"] + 1024))
        assert T >= 4 * ctas * plan["groups"] * plan["stages"]
    x, res, dy, dh = (randn(i, T, H).bfloat16() for i in range(4))
    w = (1 + 0.1 * randn(9, H)).to(torch.bfloat16 if with_dh else torch.float32)
    dh = dh if with_dh else None
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, p, seed, offset)
    assert torch.equal(h, R.dropout_fwd(x, p, seed, offset, residual=res))
    # (-0 + 0 is 0: equal to the dropout form's -0, which the norm keeps)
    y0, rstd0, _ = R.rmsnorm_fwd(torch.zeros_like(h), w, residual=h)
    assert torch.equal(y, y0) and torch.equal(rstd, rstd0)
    keep = R.dropout_fwd(torch.ones_like(x), p, seed, offset) != 0
    scale = 65536 / (65536 - round(65536 * p))
    dres0, dw0 = R.rmsnorm_bwd(dy, h, rstd, w, dh=dh)
    dw64 = sum((d.double() * q.double() * r.double()[:, None]).sum(0)
               for d, q, r in zip(dy.split(4096), h.split(4096), rstd.split(4096)))
    for det in (True, False):
        dx, dres, dw = R.rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, offset, deterministic=det,
                                             dh=dh)
        assert torch.equal(dres, dres0)
        assert not det or torch.equal(dw, dw0)
        assert ((dw.double() - dw64).abs() <= 1e-4 + 1e-4 * dw64.abs()).all()
        for part in torch.arange(T, device=DEV).split(8192):
            got, total, k = dx[part].double(), dres[part].double(), keep[part]
            assert not got[~k].any()
            # total and its product with scale are each rounded once to bf16 from FP32
            want = scale * total
            off = scale * half_step(total) * (1 + 2.0 ** -20)
            tol = off + half_step(want.abs() + off)
            assert ((got - want).abs() <= tol)[k].all()
    assert N.rmsnorm_train_device_error(reset=True) == 0


def test_allocation_through_the_dispatcher(monkeypatch):
    # what a torch without the direct allocation and stream calls runs
    x, res, dy = (randn(i, 300, 264).bfloat16() for i in range(3))
    w, b = 1 + 0.1 * randn(4, 264), randn(5, 264)

    def step():
        y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, 0.2, 6)
        g, mean, grstd = R.groupnorm_fwd(x, w, b, 8)
        return (y, rstd, h, g, R.dropout_fwd(x, 0.2, 6), R.dropout_bwd(dy, 0.2, 6),
                *R.rmsnorm_dropout_bwd(dy, h, rstd, w, 0.2, 6),
                *R.groupnorm_bwd(dy, x, mean, grstd, w, b, 8))

    want = step()
    monkeypatch.setattr(D, "_empty_strided", D._empty_strided_dispatched)
    monkeypatch.setattr(N, "_raw_stream", N._raw_stream_object)
    got = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        aside = step()
    torch.cuda.current_stream().wait_stream(side)
    for t, u, v in zip(got, aside, want):
        assert t.stride() == v.stride() and t.dtype == v.dtype
        assert torch.equal(t, v) and torch.equal(u, v)
