"""Group norm on the GPU where a value in the wrong place costs precision, or where one CTA or
cluster goes on to another sample: against the FP64 oracle, with the tolerances of
test_groupnorm_gpu.py where no other is derived here."""
from __future__ import annotations

import math

import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from oracle import groupnorm as OG
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import groupnorm as GN
from test_groupnorm_gpu import BF, DEV, EPS, FP, HF, U, case, check_bwd, check_fwd, depth, randn

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


# on chip (several stages, one stage), streamed, one thread a column, 256 lanes of it; threads
# with up to 256 places
@pytest.mark.parametrize("n,s,c,groups", [(2, 700, 64, 4), (1, 4096, 320, 32),
                                          (1, 262144, 128, 32), (1, 100000, 512, 512),
                                          (1, 20011, 2048, 1), (200, 100, 64, 8), (1, 1023, 8, 1),
                                          (2, 9, 1024, 4)])
@pytest.mark.parametrize("dtype", [BF, FP], ids=str)
@pytest.mark.parametrize("place", [0, 1, -1])
def test_one_value_far_from_the_others(n, s, c, groups, dtype, place):
    x, _, w, b = case(17, n, s, c, FP)
    x[:, place, ::c // groups] = 1000.0
    x = x.to(dtype)
    _, mean, rstd = R.groupnorm_fwd(x, w, b, groups)
    x64 = x.double()
    m64, r64 = OG.stats(x64, groups, EPS)
    # One value carries most of a group's sum of squares, and the others are near the values that
    # sums are shifted by, so nothing larger is ever added up: each of the depth's additions and
    # the products around them round within U of it; and mean's own error, squared (D U of the
    # largest value at most, over the s places that one is averaged with).
    D = depth(x, groups, False)
    big = x64.view(n, s, groups, -1).abs().amax((1, 3))
    rel = 2 * (D + 8) * U + (D * U * big * r64).square() / s + 4 * 2.0 ** -22 * m64.abs() * r64
    err = (rstd.double() - r64).abs() / r64
    assert (err <= 0.5 * rel + 2.0 ** -22).all(), (err / (0.5 * rel + 2.0 ** -22)).max()


@pytest.mark.parametrize("dtype", [BF, FP], ids=str)
@pytest.mark.parametrize("kind", ["none", "silu"])
@pytest.mark.parametrize("n,s,c,groups", [(2, 50, 64, 8), (2, 60, 40, 8), (1, 9000, 128, 32),
                                          (2, 70001, 64, 4), (700, 3, 64, 8)])
@pytest.mark.parametrize("log2", [-66, 66])
def test_gradient_of_groups_of_any_scale(n, s, c, groups, kind, dtype, log2):
    # rstd^2 passes FP32's range at either end, rstd and dx do not; groups of 1 between them
    x, dy, w, b = case(19, n, s, c, dtype)
    scale = torch.ones(c, device=DEV)
    scale.view(groups, -1)[::2] = 2.0 ** log2
    x = (x * scale).to(dtype)
    check_bwd(dy, x, w, b, groups, kind, eps=0.0)


@pytest.mark.parametrize("c,groups", [(40, 8), (64, 4), (24, 8)])
@pytest.mark.parametrize("s", [60, 3000, 70001])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=str)
def test_nan_and_infinity_leave_the_other_groups_their_bits(c, groups, s, kind, dtype):
    x, dy, w, b = case(23, 2, s, c, dtype)
    per = c // groups
    clean = R.groupnorm_fwd(x, w, b, groups, EPS, kind)
    gclean = R.groupnorm_bwd(dy, x, clean[1], clean[2], w, b, groups, kind)
    bad = x.clone()
    bad[1, s // 2, 2 * per] = float("nan")
    bad[0, 0, per - 1] = float("-inf")
    y, mean, rstd = R.groupnorm_fwd(bad, w, b, groups, EPS, kind)
    dx, dw, db = R.groupnorm_bwd(dy, bad, mean, rstd, w, b, groups, kind)
    hit = torch.zeros(2, groups, dtype=torch.bool, device=DEV)
    hit[1, 2] = hit[0, 0] = True
    assert torch.equal(~rstd.isfinite(), hit)
    wide = hit.repeat_interleave(per, 1)[:, None].expand(x.shape)
    cols = hit.any(0).repeat_interleave(per)
    assert y[wide].isnan().all() and dx[wide].isnan().all() and dw[cols].isnan().all()
    for got, want in ((y[~wide], clean[0][~wide]), (dx[~wide], gclean[0][~wide]),
                      (dw[~cols], gclean[1][~cols]), (db[~cols], gclean[2][~cols])):
        assert torch.equal(got, want)


# clusters of 2, 4 and 8 CTAs that take 1.5 to 8 samples each
FWD_CLUSTERS = [(HF, 114, 6, 2296, 2), (BF, 124, 6, 2344, 2), (FP, 25, 22, 2104, 2),
                (BF, 75, 342, 72, 6), (FP, 11, 14, 2152, 2), (HF, 37, 622, 72, 8),
                (BF, 64, 8, 2168, 1)]
BWD_CLUSTERS = [(FP, 160, 3, 1576, 1), (FP, 212, 221, 56, 8), (BF, 52, 4, 2104, 2),
                (FP, 156, 7, 1384, 173), (FP, 11, 11, 2104, 8), (HF, 37, 622, 72, 8),
                (BF, 119, 8, 2128, 1)]


def several_samples_a_cluster(dtype, n, s, c, groups, bwd):
    p = N.groupnorm_train_launch_plan(GN._DTYPES[dtype], n, s, c, groups, bwd)
    return p["on_chip"] and p["cluster_ctas"] > 1 and p["ctas"] < p["units"] * p["cluster_ctas"]


@pytest.mark.parametrize("dtype,n,s,c,groups", FWD_CLUSTERS, ids=str)
def test_clusters_go_on_to_further_samples_forward(dtype, n, s, c, groups):
    assert several_samples_a_cluster(dtype, n, s, c, groups, 0)
    x, _, w, b = case(29, n, s, c, dtype)
    got = check_fwd(x, w, b, groups, "silu")
    for _ in range(3):
        again = R.groupnorm_fwd(x, w, b, groups, EPS, "silu")
        assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype,n,s,c,groups", BWD_CLUSTERS, ids=str)
def test_clusters_go_on_to_further_samples_backward(dtype, n, s, c, groups):
    assert several_samples_a_cluster(dtype, n, s, c, groups, 1)
    x, dy, w, b = case(31, n, s, c, dtype)
    got = check_bwd(dy, x, w, b, groups, "silu")
    mean, rstd = (t.float() for t in OG.stats(x.double(), groups, EPS))
    for _ in range(3):
        again = R.groupnorm_bwd(dy, x, mean, rstd, w, b, groups, "silu")
        assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_forms_of_many_small_samples():
    # forward on chip, backward streamed in one piece a sample
    p = [N.groupnorm_train_launch_plan(N.GROUPNORM_FP32, 700, 300, 64, 8, d) for d in (0, 1)]
    assert p[0]["on_chip"] and not p[1]["on_chip"] and p[1]["chunks"] == 1


# one to three places a sample and every channel in one slab
@pytest.mark.parametrize("dtype,n,s,c,groups", [
    (BF, 3000, 1, 2048, 1), (HF, 700, 2, 2048, 1), (BF, 333, 3, 2048, 1), (BF, 1200, 1, 4096, 1),
    (HF, 500, 2, 4096, 1), (BF, 401, 3, 4096, 1), (BF, 700, 1, 3000, 8), (FP, 900, 1, 2048, 1),
    (BF, 64, 1, 4096, 1), (BF, 5, 3, 4088, 8)], ids=str)
def test_few_places_of_wide_slabs(dtype, n, s, c, groups):
    x, dy, w, b = case(37, n, s, c, dtype)
    check_fwd(x, w, b, groups, "silu")
    got = check_bwd(dy, x, w, b, groups, "silu")
    mean, rstd = (t.float() for t in OG.stats(x.double(), groups, EPS))
    again = R.groupnorm_bwd(dy, x, mean, rstd, w, b, groups, "silu")
    assert all(torch.equal(p, q) for p, q in zip(got, again))


# sequences of pieces that share a row of sums, and one place a sample on chip
@pytest.mark.parametrize("dtype,n,s,c", [(BF, 1300, 2, 2048), (HF, 401, 3, 4096), (BF, 900, 1, 4096)],
                         ids=str)
def test_few_places_of_wide_slabs_captured_and_side_by_side(dtype, n, s, c):
    cases = [case(41 + i, n, s, c, dtype) for i in range(2)]

    def step(x, dy, w, b):
        _, mean, rstd = R.groupnorm_fwd(x, w, b, 1, act="silu")
        return R.groupnorm_bwd(dy, x, mean, rstd, w, b, 1, "silu")

    want = [step(*args) for args in cases]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for args in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(*args))
    for _ in range(4):                            # each finds the last replay's sums in its workspace
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(p, q))
    # one infinite gradient: its channel's sums are infinite, the other channels' as before
    x, dy, w, b = cases[0]
    _, mean, rstd = R.groupnorm_fwd(x, w, b, 1)
    clean = R.groupnorm_bwd(dy, x, mean, rstd, w, b, 1)
    dy[n // 2, s - 1, 5] = float("inf")
    dx, dw, db = R.groupnorm_bwd(dy, x, mean, rstd, w, b, 1)
    assert db[5] == float("inf") and dw[5].isinf()
    rest = torch.arange(c, device=DEV) != 5
    assert torch.equal(dw[rest], clean[1][rest]) and torch.equal(db[rest], clean[2][rest])
    rows = torch.arange(n, device=DEV) != n // 2
    assert torch.equal(dx[rows], clean[0][rows])
