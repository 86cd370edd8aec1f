"""The group norm entry points on the GPU against the FP64 oracle (oracle/groupnorm.py), element
by element.

Tolerances, from the roundings (U = 2^-24, u half a step of the output type).  D bounds the
additions a value passes through on its way into a sum (depth(), from the launch plan): a
thread's places, the CTA's, the cluster's and the chunks'.
  mean   D U times the largest |x| of the group (each partial sum of a mean is within that)
  var    a column's M2 = sum d^2 - (sum d)^2 / n with d = x - K: relative to M2_c + 2 n d^2,
         (D + 8) U each, so with k = max |x - mean|^2 / var: (D + 8) (1 + 2 k) U; about a
         CTA's rounded mean, 2^-22 |mean| / sigma twice, and mean's own error squared
  z      |w| (rstd tol_mean + |x - mean| tol_rstd) + 2^-22 (|xhat w| + |b|)
  act    slopes at most 1.13; the sigmoid's FP32 roundings 2^-22 (8 + |z|) relative (exp's
         argument carries |z| U), 2^-61 |z| absolute, erf's 2^-22 |z| absolute
  dz     from the given mean and rstd: z's roundings times the largest curvature (0.8), the
         slope's roundings
  dx     the errors of g through both means, D U of each mean, the final roundings
  dw, db the errors of dz, D U of the sums of absolute terms, one rounding to FP32
"""
from __future__ import annotations

import math

import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from oracle import groupnorm as OG
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import groupnorm as GN

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
EPS = 1e-5
BF, FP, HF = torch.bfloat16, torch.float32, torch.float16


def randn(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV)


def half_step(v, dtype):
    """Half a step of dtype at the values v (FP32: its one rounding)."""
    info = torch.finfo(dtype)
    return v.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2


def depth(x, groups, bwd):
    n, s, c = x.shape
    p = N.groupnorm_train_launch_plan(GN._DTYPES[x.dtype], n, s, c, groups, bwd)
    lanes = max(1, p["threads"] * (16 // x.element_size()) // p["channels"])
    if p["on_chip"]:
        rows, chunks = -(-s // p["cluster_ctas"]), 1
    else:
        chunks = p["chunks"]
        rows = -(-s // chunks)
    # a thread's places (at least half the lanes the plan has threads for), four lanes of a
    # column at a time, eight columns of a group, 32 chunks; the trees between
    places = rows // max(1, (lanes + 1) // 2) + 2
    return places + lanes / 4 + 3 + c // groups / 8 + 4 + 4 + chunks / 32 + 6


def case(seed, n, s, c, dtype, wb=FP, offset=0.0):
    x = (randn(seed, n, s, c) + 0.5 * randn(seed + 1, c) + offset).to(dtype)
    dy = randn(seed + 2, n, s, c).to(dtype)
    w = (1 + 0.1 * randn(seed + 3, c)).to(wb)
    b = (0.1 * randn(seed + 4, c)).to(wb)
    return x, dy, w, b


def act_error(z, y, kind):
    if kind == "silu":
        return 2.0 ** -22 * (8 + z.abs()) * y.abs() + 2.0 ** -61 * z.abs()
    if kind == "gelu":
        return 2.0 ** -22 * z.abs()
    return 0.0


def slope_error(z, kind):
    return 0.0 if kind == "none" else 2.0 ** -21 * (4 + z.abs())


def check_fwd(x, w, b, groups, kind, eps=EPS, got=None):
    y, mean, rstd = R.groupnorm_fwd(x, w, b, groups, eps, kind) if got is None else got
    n, c = x.shape[0], x.shape[-1]
    assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
    x64 = x.double().reshape(n, -1, c)
    w64, b64 = w.double(), b.double()
    eps = float(torch.tensor(eps, dtype=FP))
    y64, m64, r64 = OG.fwd(x64, w64, b64, groups, eps, kind)
    D = depth(x64.to(x.dtype), groups, False)
    grouped = x64.view(n, x64.shape[1], groups, -1)
    dev = (grouped - m64[:, None, :, None]).abs().amax((1, 3))
    var = 1 / r64.square() - eps
    sigma = var.clamp(min=1e-300).sqrt()
    tol_mean = D * U * grouped.abs().amax((1, 3))
    rel_var = ((D + 8) * (1 + 2 * dev.square() / var.clamp(min=1e-300)) * U
               + 4 * 2.0 ** -22 * m64.abs() / sigma + (tol_mean / sigma).square())
    tol_rstd = r64 * (0.5 * rel_var * var / (var + eps) + 2.0 ** -22)
    assert ((mean.double() - m64).abs() <= tol_mean).all()
    assert ((rstd.double() - r64).abs() <= tol_rstd).all()
    xm = x64 - OG.wide(m64, c)
    xw = xm * OG.wide(r64, c) * w64
    z = xw + b64
    ez = (w64.abs() * (OG.wide(r64 * tol_mean, c) + xm.abs() * OG.wide(tol_rstd, c))
          + 2.0 ** -22 * (xw.abs() + b64.abs()))
    e = 1.13 * ez + act_error(z, y64, kind)
    err = (y.double().reshape(n, -1, c) - y64).abs()
    assert (err <= e + half_step(y64.abs() + e, x.dtype)).all(), (err / (e + half_step(
        y64.abs() + e, x.dtype))).max()
    return y, mean, rstd


def check_bwd(dy, x, w, b, groups, kind, eps=EPS):
    n, c = x.shape[0], x.shape[-1]
    x64, dy64 = x.double().reshape(n, -1, c), dy.double().reshape(n, -1, c)
    w64, b64 = w.double(), b.double()
    mean, rstd = (t.float() for t in OG.stats(x64, groups, eps))
    dx, dw, db = R.groupnorm_bwd(dy, x, mean, rstd, w, b, groups, kind)
    m64, r64 = mean.double(), rstd.double()
    dx64, dw64, db64 = OG.bwd(dy64, x64, m64, r64, w64, b64, groups, kind)
    D = depth(x64.to(x.dtype), groups, True)
    rw = OG.wide(r64, c)
    xhat = (x64 - OG.wide(m64, c)) * rw
    z = xhat * w64 + b64
    dz = dy64 * OG.slope(z, kind)
    g = dz * w64
    ez = 2.0 ** -22 * ((xhat * w64).abs() + b64.abs())
    edz = (dy64.abs() * (0.8 * ez + slope_error(z, kind)) if kind != "none" else 0.0) \
        + 2.0 ** -22 * dz.abs()
    eg = edz * w64.abs()
    gm = lambda t: OG.group_mean(t, groups)  # noqa: E731
    e = rw * (eg + gm(eg) + xhat.abs() * gm(eg * xhat.abs())
              + 2.0 ** -21 * (g.abs() + gm(g).abs() + (xhat * gm(g * xhat)).abs())
              + (D + 8) * U * (gm(g.abs()) + xhat.abs() * gm((g * xhat).abs())))
    err = (dx.double().reshape(n, -1, c) - dx64).abs()
    tol = e + half_step(dx64.abs() + e, x.dtype)
    assert dx.shape == x.shape and dx.dtype == x.dtype and (err <= tol).all(), (err / tol).max()
    for got, want, terms, edges in ((dw, dw64, dz * xhat, edz * xhat.abs()), (db, db64, dz, edz)):
        tol = edges.sum((0, 1)) + (D + 8) * U * terms.abs().sum((0, 1)) + 2.0 ** -23 * want.abs()
        assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol).max()
    return dx, dw, db


# (N, S, C, groups): one place, one channel a group, groups that split vectors (odd and even),
# one group, wide groups, clusters of 2, 4 and 8, ragged places
SHAPES = [(1, 1, 64, 1), (3, 1, 256, 4), (2, 7, 8, 1), (2, 37, 64, 64), (3, 33, 40, 8),
          (2, 130, 24, 8), (5, 50, 320, 32), (1, 3, 4088, 8), (2, 9, 2048, 1), (2, 64, 1280, 32),
          (7, 257, 96, 6), (1, 1023, 640, 32), (2, 1500, 72, 8), (1, 4096, 320, 32),
          (1, 9000, 128, 32), (300, 5, 64, 8)]
# streamed: samples past a cluster's shared memory, several turns, wide slabs
LARGE = [(1, 70001, 64, 4), (13, 70001, 64, 4), (1, 20011, 520, 8), (1, 301, 2048, 1),
         (1, 350001, 128, 32), (2, 500, 4096, 1), (3, 411, 4088, 8)]


def too_wide(dtype, c, groups):
    """Whether the fewest groups that make whole 16-byte vectors hold more than 512 of them."""
    ev = 8 if dtype != FP else 4
    width = c // groups
    return width * (ev // math.gcd(width, ev)) // ev > 512


@pytest.mark.parametrize("n,s,c,groups", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=str)
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_forward(n, s, c, groups, dtype, kind):
    x, _, w, b = case(s + c, n, s, c, dtype, FP if kind == "silu" else dtype)
    if too_wide(dtype, c, groups):
        with pytest.raises(N.RmsnError, match="unsupported"):
            R.groupnorm_fwd(x, w, b, groups)
        return
    got = check_fwd(x, w, b, groups, kind)
    again = R.groupnorm_fwd(x, w, b, groups, EPS, kind)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("n,s,c,groups", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=str)
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_backward(n, s, c, groups, dtype, kind):
    x, dy, w, b = case(s + c, n, s, c, dtype, FP if kind == "silu" else dtype)
    if too_wide(dtype, c, groups):
        with pytest.raises(N.RmsnError, match="unsupported"):
            R.groupnorm_bwd(dy, x, torch.zeros(n, groups, device=DEV),
                            torch.ones(n, groups, device=DEV), w, b, groups)
        return
    check_bwd(dy, x, w, b, groups, kind)


@pytest.mark.parametrize("n,s,c,groups", LARGE)
@pytest.mark.parametrize("dtype", [BF, FP], ids=str)
def test_streamed(n, s, c, groups, dtype):
    if too_wide(dtype, c, groups):
        pytest.skip("more than 512 vectors a slab")
    x, dy, w, b = case(n + s, n, s, c, dtype)
    plans = [N.groupnorm_train_launch_plan(GN._DTYPES[dtype], n, s, c, groups, d) for d in (0, 1)]
    assert not plans[1]["on_chip"]
    if n > 10:  # several turns
        assert not plans[0]["on_chip"] and plans[0]["units"] < n * c // plans[0]["channels"]
    if s > 300000:  # a sample too large for one turn
        assert plans[1]["units"] < c // plans[1]["channels"]
    got = check_fwd(x, w, b, groups, "silu")
    grads = check_bwd(dy, x, w, b, groups, "silu")
    assert all(torch.equal(p, q) for p, q in zip(got, R.groupnorm_fwd(x, w, b, groups, EPS, "silu")))
    mean, rstd = (t.float() for t in OG.stats(x.double(), groups, EPS))
    again = R.groupnorm_bwd(dy, x, mean, rstd, w, b, groups, "silu")
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


@pytest.mark.parametrize("s", [50, 5000, 70001])
@pytest.mark.parametrize("dtype,offset", [(FP, 1000.0), (FP, -30000.0), (BF, 100.0), (HF, 200.0)])
def test_mean_far_from_zero(s, dtype, offset):
    x, dy, w, b = case(7, 2, s, 64, dtype, offset=offset)
    _, _, rstd = check_fwd(x, w, b, 4, "silu")
    # (the derived tolerance grows with the mean; the shifted sums do better than it says)
    want = OG.stats(x.double(), 4, EPS)[1]
    assert ((rstd.double() - want).abs() <= 2e-3 * want).all()
    check_bwd(dy, x, w, b, 4, "silu")


def test_constant_groups():
    x = torch.full((2, 100, 64), 0.1, device=DEV)
    x[1, :, :16] = 0.0
    w, b = 1 + 0.1 * randn(1, 64), randn(2, 64)
    y, mean, rstd = R.groupnorm_fwd(x, w, b, 4)
    # mean is within a few roundings of 0.1, and nothing else differs from it
    off = 64 * U * 0.1
    assert ((mean - x[:, 0, ::16]).abs() <= off).all()
    assert ((rstd.double() - EPS ** -0.5).abs() <= EPS ** -0.5 * (off * off / EPS + 2.0 ** -21)).all()
    assert ((y - b).abs() <= 1.5 * off * EPS ** -0.5 + 2.0 ** -22 * b.abs()).all()
    assert torch.equal(y[1, :, :16], b[:16].expand(100, 16))


@pytest.mark.parametrize("c,groups", [(40, 8), (64, 4)])
@pytest.mark.parametrize("s", [60, 3000, 70001])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_a_group_with_nan_or_infinity_keeps_it(c, groups, s, kind):
    # groups of five channels share 16-byte vectors and pairs with their neighbours
    x, dy, w, b = case(3, 2, s, c, BF)
    clean = R.groupnorm_fwd(x, w, b, groups, EPS, kind)
    gclean = R.groupnorm_bwd(dy, x, clean[1], clean[2], w, b, groups, kind)
    bad = x.clone()
    per = c // groups
    bad[1, s // 2, 2 * per] = float("nan")
    bad[0, s // 3, 5 * per - 1 if groups > 4 else 0] = float("inf")
    y, mean, rstd = R.groupnorm_fwd(bad, w, b, groups, EPS, kind)
    dx, dw, db = R.groupnorm_bwd(dy, bad, mean, rstd, w, b, groups, kind)
    hit = torch.zeros(2, groups, dtype=torch.bool, device=DEV)
    hit[1, 2] = True
    hit[0, 4 if groups > 4 else 0] = True
    wide = hit.repeat_interleave(per, 1)[:, None].expand(x.shape)
    assert torch.equal(~rstd.isfinite(), hit)
    assert y[wide].isnan().all() and dx[wide].isnan().all()
    cols = hit.any(0).repeat_interleave(per)
    assert dw[cols].isnan().all()
    for got, want in ((y[~wide], clean[0][~wide]), (dx[~wide], gclean[0][~wide]),
                      (dw[~cols], gclean[1][~cols]), (db[~cols], gclean[2][~cols])):
        if kind == "silu" and per % 2:
            # two channels of a pair share a reciprocal: a neighbour's value moves FP32
            # roundings (of 2^-22 at most, summed for dw and db), never more
            assert (got - want).abs().max() <= 2.0 ** -7 * want.abs().max()
            assert got.isfinite().all()
        else:
            assert torch.equal(got, want)


def test_large_activations_saturate():
    # z in the hundreds and far below -62 ln 2: the sigmoid's ends
    x = torch.zeros(1, 64, 16, device=DEV, dtype=BF)
    x[0, ::2] = 1.0
    w = torch.tensor([200.0, 30.0] * 8, device=DEV)
    b = torch.zeros(16, device=DEV)
    dy = randn(3, 1, 64, 16).to(BF)
    for kind in ("silu", "gelu"):
        check_fwd(x, w, b, 2, kind)
        check_bwd(dy, x, w, b, 2, kind)
        check_fwd(x.float(), w, b, 2, kind)
        check_bwd(dy.float(), x.float(), w, b, 2, kind)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, FP], ids=str)
def test_activations_far_out(dtype, kind):
    # z = +-w with w past anything the exponentials hold: act is z or 0, its slope 1 or 0
    x = torch.zeros(1, 64, 16, device=DEV, dtype=dtype)
    x[0, ::2] = 1.0
    w = torch.full((16,), 2.0 ** 99, device=DEV)
    b = torch.zeros(16, device=DEV)
    dy = torch.ones(1, 64, 16, device=DEV, dtype=dtype)
    y, mean, rstd = R.groupnorm_fwd(x, w, b, 2, act=kind)
    assert not y[0, 1::2].any()
    z = 2.0 ** 99 * 0.5 * rstd[0, 0].double().item()
    tol = z * (2.0 ** -21 + torch.finfo(dtype).eps / 2)
    assert ((y[0, ::2].double() - z).abs() <= tol).all()
    dx, dw, db = R.groupnorm_bwd(dy, x, mean, rstd, w, b, 2, kind)
    # dz is dy on the places with z > 0: 32 ones a channel, and xhat = 0.5 rstd there
    assert torch.equal(db, torch.full_like(db, 32.0))
    want = 32 * 0.5 * rstd[0, 0].double()
    assert ((dw.double() - want).abs() <= want * 2.0 ** -18).all()
    assert dx.isfinite().all()


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=str)
def test_an_overflowing_norm_is_infinite(dtype, kind):
    x = torch.zeros(1, 64, 16, device=DEV, dtype=dtype)
    x[0, ::2] = 1.0
    w, b = torch.full((16,), 3e38, device=DEV), torch.zeros(16, device=DEV)
    y, _, _ = R.groupnorm_fwd(x, w, b, 2, act=kind)
    assert torch.equal(y[0, ::2], torch.full_like(y[0, ::2], float("inf")))


@pytest.mark.parametrize("dtype", [BF, HF, FP], ids=str)
def test_gelu_along_its_argument(dtype):
    # w = 0: z is b, one value a channel; with dy = 1 db is the slope, in FP32
    c, groups = 4096, 64
    z = torch.linspace(-12, 12, c, device=DEV)
    x, w = randn(1, 1, 1, c).to(dtype), torch.zeros(c, device=DEV)
    y, mean, rstd = R.groupnorm_fwd(x, w, z, groups, act="gelu")
    dx, dw, db = R.groupnorm_bwd(torch.ones_like(x), x, mean, rstd, w, z, groups, "gelu")
    z64 = z.double()
    y64, a = OG.act(z64, "gelu"), z64.abs()
    # Phi(-a) within 1.5e-7, below a = 5 also within 2e-5 of itself; the rounded exponent adds
    # 2^-23 z^2 / 2 and the approximate functions 2^-21 (FP32: erf's 2^-22)
    q = 0.5 * torch.erfc(a / math.sqrt(2))
    tail = torch.where(a < 5, q * (2e-5 + 2.0 ** -23 * a * a / 2 + 2.0 ** -21), q + 1.5e-7)
    dq = torch.full_like(q, 2.0 ** -22) if dtype == FP else tail.clamp(max=2e-7)
    e = a * dq + 2.0 ** -23 * y64.abs()
    assert ((y[0, 0].double() - y64).abs() <= e + half_step(y64.abs() + e, dtype)).all()
    # the slope: 1 - Phi's rounding, phi's argument, and dq
    assert ((db.double() - OG.slope(z64, "gelu")).abs() <= 2e-7 + 2.0 ** -21).all()
    assert not dx.any()


def test_strided_input():
    wide = randn(1, 3, 40, 256).to(BF)
    w, b = 1 + 0.1 * randn(2, 64), 0.1 * randn(3, 64)
    dy = randn(4, 3, 40, 64).to(BF)
    for x in (wide[..., 64:128], wide[:, 3:35, 8:72], wide[:, ::2, 128:192], wide[::2, :, :64],
              wide.transpose(0, 1)[..., :64]):
        d = randn(5, *x.shape).to(BF)
        y, mean, rstd = R.groupnorm_fwd(x, w, b, 8, act="silu")
        got = R.groupnorm_bwd(d, x, mean, rstd, w, b, 8, "silu")
        want = R.groupnorm_fwd(x.contiguous(), w, b, 8, act="silu")
        assert torch.equal(y, want[0]) and torch.equal(mean, want[1])
        for p, q in zip(got, R.groupnorm_bwd(d, x.contiguous(), mean, rstd, w, b, 8, "silu")):
            assert torch.equal(p, q)
    # spatial axes merge; a channels_last image is its permuted view
    img = randn(6, 2, 64, 6, 7).to(BF).to(memory_format=torch.channels_last)
    y, _, _ = R.groupnorm_fwd(img.permute(0, 2, 3, 1), w, b, 8)
    flat = img.permute(0, 2, 3, 1).reshape(2, 42, 64)
    assert y.shape == (2, 6, 7, 64)
    assert torch.equal(y.view(2, 42, 64), R.groupnorm_fwd(flat, w, b, 8)[0])
    assert torch.equal(R.groupnorm_bwd(dy.transpose(0, 1).contiguous().transpose(0, 1),
                                       wide[..., :64], *R.groupnorm_fwd(wide[..., :64], w, b, 8)[1:],
                                       w, b, 8)[0],
                       R.groupnorm_bwd(dy, wide[..., :64].contiguous(),
                                       *R.groupnorm_fwd(wide[..., :64], w, b, 8)[1:], w, b, 8)[0])


def test_refusals():
    x = randn(1, 2, 6, 5, 64).to(BF)
    w, b = torch.ones(64, device=DEV), torch.zeros(64, device=DEV)
    mean, rstd = torch.zeros(2, 8, device=DEV), torch.ones(2, 8, device=DEV)
    for match, call in [
            ("groups", lambda: R.groupnorm_fwd(x, w, b, 7)),
            ("groups", lambda: R.groupnorm_fwd(x, w, b, 0)),
            ("act", lambda: R.groupnorm_fwd(x, w, b, 8, act="tanh")),
            ("shape", lambda: R.groupnorm_fwd(x, w[:32], b, 8)),
            ("places", lambda: R.groupnorm_fwd(x[:, :0], w, b, 8)),
            ("channels last", lambda: R.groupnorm_fwd(x.transpose(1, 3), w[:6], b[:6], 3)),
            ("merge", lambda: R.groupnorm_fwd(x[:, :, :3], w, b, 8)),
            ("dy", lambda: R.groupnorm_bwd(x[:1], x, mean, rstd, w, b, 8)),
            ("dy", lambda: R.groupnorm_bwd(x.float(), x, mean, rstd, w, b, 8)),
            ("mean", lambda: R.groupnorm_bwd(x, x, mean[:, :4], rstd, w, b, 8)),
            ("rstd", lambda: R.groupnorm_bwd(x, x, mean, rstd.double(), w, b, 8)),
            ("one device", lambda: R.groupnorm_fwd(x, w.cpu(), b, 8))]:
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(TypeError, match="w and b"):
        R.groupnorm_fwd(x, w, b.half(), 8)
    with pytest.raises(TypeError, match="x must"):
        R.groupnorm_fwd(x.double(), w, b, 8)
    with pytest.raises(N.RmsnError):              # places 8 bytes apart from 16-byte steps
        R.groupnorm_fwd(randn(1, 2, 6, 68).to(BF)[..., :64], w, b, 8)
    with pytest.raises(N.RmsnError):
        R.groupnorm_fwd(randn(1, 2, 6, 12).to(BF), w[:12], b[:12], 3)


def test_no_samples():
    x = torch.empty(0, 5, 64, device=DEV, dtype=BF)
    w, b = torch.ones(64, device=DEV), torch.zeros(64, device=DEV)
    y, mean, rstd = R.groupnorm_fwd(x, w, b, 8)
    assert y.shape == x.shape and mean.shape == (0, 8)
    dx, dw, db = R.groupnorm_bwd(x, x, mean, rstd, w, b, 8)
    assert dx.shape == x.shape and not dw.any() and not db.any()
    assert R.groupnorm_fwd(x[:, :0], w, b, 8)[0].shape == (0, 0, 64)


def test_many_samples_on_chip():
    # every cluster takes several samples: staging and running totals are used again
    x, dy, w, b = case(11, 6000, 3, 64, BF)
    p = N.groupnorm_train_launch_plan(N.GROUPNORM_BF16, 6000, 3, 64, 8, 1)
    assert p["on_chip"] and p["ctas"] < 6000
    check_fwd(x, w, b, 8, "silu")
    check_bwd(dy, x, w, b, 8, "silu")
    x, dy, w, b = case(12, 700, 300, 64, FP)
    assert N.groupnorm_train_launch_plan(N.GROUPNORM_FP32, 700, 300, 64, 8, 1)["cluster_ctas"] >= 1
    check_fwd(x, w, b, 8, "silu")
    check_bwd(dy, x, w, b, 8, "silu")


@pytest.mark.parametrize("wb", [BF, FP])
def test_autograd(wb):
    x, dy, w, b = case(5, 2, 300, 96, BF, wb)
    for t in (x, w, b):
        t.requires_grad_()
    y = R.groupnorm_train(x, w, b, 6, act="silu")
    y.backward(dy)
    d = [t.detach() for t in (x, w, b)]
    y0, mean, rstd = R.groupnorm_fwd(*d, 6, act="silu")
    dx, dw, db = R.groupnorm_bwd(dy, d[0], mean, rstd, d[1], d[2], 6, "silu")
    assert torch.equal(y, y0) and torch.equal(x.grad, dx)
    assert torch.equal(w.grad, dw.to(wb)) and torch.equal(b.grad, db.to(wb))


@pytest.mark.parametrize("s", [100, 3000, 70001])
def test_captured_and_replayed(s):
    x, dy, w, b = case(9, 2, s, 64, BF)

    def step():
        y, mean, rstd = R.groupnorm_fwd(x, w, b, 4, act="silu")
        return (y, mean, rstd) + R.groupnorm_bwd(dy, x, mean, rstd, w, b, 4, "silu")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (1, 2):                          # new inputs in the same buffers
        x.copy_(randn(seed, 2, s, 64))
        dy.copy_(randn(seed + 10, 2, s, 64))
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_two_streams_at_once():
    cases = [case(20 + i, 2, 70001, 64, BF) for i in range(2)]
    want = [R.groupnorm_fwd(x, w, b, 4)[0] for x, _, w, b in cases]
    grads = [R.groupnorm_bwd(dy, x, *R.groupnorm_fwd(x, w, b, 4)[1:], w, b, 4)
             for x, dy, w, b in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    out = [[], []]
    for _ in range(5):
        for i, (x, dy, w, b) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                y, mean, rstd = R.groupnorm_fwd(x, w, b, 4)
                out[i].append((y,) + R.groupnorm_bwd(dy, x, mean, rstd, w, b, 4))
    torch.cuda.synchronize()
    for i in range(2):
        for got in out[i]:
            assert torch.equal(got[0], want[i])
            assert all(torch.equal(p, q) for p, q in zip(got[1:], grads[i]))


def test_two_graphs_at_once():
    # each has its own workspace; the streamed form's grids wait for each other's SMs at most
    cases = [case(60 + i, 2, 70001, 64, BF) for i in range(2)]

    def step(x, dy, w, b):
        y, mean, rstd = R.groupnorm_fwd(x, w, b, 4, act="silu")
        return (y,) + R.groupnorm_bwd(dy, x, mean, rstd, w, b, 4, "silu")

    want = [step(*c) for c in cases]
    torch.cuda.synchronize()
    graphs, got, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(step(*c))
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(p, q))


@pytest.mark.parametrize("n,s", [(2, 300), (6000, 3), (2, 70001)])
def test_an_infinite_gradient_stays_infinite_in_its_sums(n, s):
    # one channel's gradient overflows: its db is infinite, dw too, the other channels' as before
    x, dy, w, b = case(70, n, s, 64, FP)
    _, mean, rstd = R.groupnorm_fwd(x, w, b, 8)
    want = R.groupnorm_bwd(dy, x, mean, rstd, w, b, 8)
    dy[0, 1, 5] = float("inf")
    got = R.groupnorm_bwd(dy, x, mean, rstd, w, b, 8)
    xhat = (x[0, 1, 5] - mean[0, 0]).sign()
    assert got[2][5] == float("inf") and got[1][5] == float("inf") * xhat
    rest = torch.arange(64, device=DEV) != 5
    for g, e in zip(got[1:], want[1:]):
        assert torch.equal(g[rest], e[rest])


def test_gradient_at_any_address():
    x, dy, w, b = case(71, 2, 50, 64, BF)
    _, mean, rstd = R.groupnorm_fwd(x, w, b, 8)
    off = torch.cat([dy.new_zeros(3), dy.flatten()])[3:].view_as(dy)
    assert off.is_contiguous() and off.data_ptr() % 16
    for p, q in zip(R.groupnorm_bwd(off, x, mean, rstd, w, b, 8),
                    R.groupnorm_bwd(dy, x, mean, rstd, w, b, 8)):
        assert torch.equal(p, q)
    with pytest.raises(N.RmsnError):
        R.groupnorm_fwd(off, w, b, 8)


def test_block_of_all_the_operators():
    """A residual block as a training step runs it, eagerly and captured: group norm with SiLU,
    dropout, a projection, dropout with the residual RMSNorm; gradients against the same block
    from the oracles' formulas in float64."""
    from oracle import dropout as OD
    n, s, c, groups, p, seed = 2, 130, 64, 8, 0.25, 1234
    x, dy, w, b = case(31, n, s, c, BF)
    dh = randn(40, n, s, c).to(BF)
    proj = (randn(41, c, c) / 8).to(BF)
    w2 = 1 + 0.1 * randn(42, c)
    leaves = [t.requires_grad_() for t in (x, w, b, proj, w2)]

    def block():
        a = R.groupnorm_train(x, w, b, groups, act="silu")
        z = R.dropout_train(a, p, seed, 0) @ proj
        y, h = R.rmsnorm_dropout_train(z.view(-1, c), x.view(-1, c), w2, p, seed, 1)
        return y, h

    def grads():
        y, h = block()
        return torch.autograd.grad((y, h), leaves, (dy.view(-1, c), dh.view(-1, c)))

    got = grads()
    # float64, by torch's autograd through the formulas, masks from the oracle
    x6, w6, b6, p6, v6 = (t.detach().double().requires_grad_() for t in leaves)
    keep = [torch.from_numpy(OD.keep(n * s * c, p, seed, i)).to(DEV).view(n, s, c).double()
            * OD.scale(p) for i in (0, 1)]
    a6 = OG.fwd(x6, w6, b6, groups, EPS, "silu")[0]
    h6 = x6 + (a6 * keep[0]) @ p6 * keep[1]
    y6 = h6 / torch.sqrt(h6.square().mean(2, keepdim=True) + 1e-6) * v6
    want = torch.autograd.grad((y6, h6), (x6, w6, b6, p6, v6), (dy.double(), dh.double()))
    # every bf16 tensor between (a, dropout, z, h, y and their gradients) is rounded once, by
    # 2^-8 at most; twelve of them, added up in the 2-norm through operators of norm near one
    for g, e in zip(got, want):
        assert (g.double() - e).norm() <= 12 * 2.0 ** -8 * e.norm()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = grads()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, e) for g, e in zip(captured, got))


def test_elements_past_32_bits():
    # 3.2e9 elements (and byte offsets past 2^32): the last sample as when it is alone
    n, s, c, groups = 3, 1 << 20, 1024, 32
    x = torch.empty(n, s, c, dtype=BF, device=DEV).normal_()
    dy = torch.empty_like(x).normal_()
    w, b = 1 + 0.1 * randn(1, c), 0.1 * randn(2, c)
    y, mean, rstd = R.groupnorm_fwd(x, w, b, groups, act="silu")
    y1, mean1, rstd1 = R.groupnorm_fwd(x[2:], w, b, groups, act="silu")
    dx, dw, db = R.groupnorm_bwd(dy, x, mean, rstd, w, b, groups, "silu")
    parts = [R.groupnorm_bwd(dy[i:i + 1], x[i:i + 1], mean[i:i + 1], rstd[i:i + 1], w, b, groups,
                             "silu") for i in range(n)]
    # the same sums in other orders: 2^-24 a step, well under a bf16 rounding; an output differs
    # where that tips it, by one bf16 step (2^-7 of the value, 2^-20 of the scale near zero)
    assert (mean[2:] - mean1).abs().max() < 1e-6 and (rstd[2:] / rstd1 - 1).abs().max() < 1e-5
    for at in (0, s // 2, s - 4096):
        part = slice(at, at + 4096)
        for got, want in ((y[2, part], y1[0, part]), (dx[2, part], parts[2][0][0, part])):
            got, want = got.float(), want.float()
            assert ((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -20).all()
    for got, i in ((dw, 1), (db, 2)):
        want = sum(p[i].double() for p in parts)
        # n * s terms of about one each: sums of absolute values near n s, in 2^-24 steps
        assert (got.double() - want).abs().max() < 64 * U * n * s


def test_strides_past_32_bits():
    buf = torch.empty((1 << 32) + 64 * 64, dtype=BF, device=DEV)
    x = buf.as_strided((2, 64, 64), (1 << 32, 64, 1))
    x.copy_(randn(1, 2, 64, 64))
    w, b = 1 + 0.1 * randn(2, 64), 0.1 * randn(3, 64)
    got = R.groupnorm_fwd(x, w, b, 8)
    want = R.groupnorm_fwd(x.contiguous(), w, b, 8)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for p, q in zip(R.groupnorm_bwd(want[0], x, *got[1:], w, b, 8),
                    R.groupnorm_bwd(want[0], x.contiguous(), *got[1:], w, b, 8)):
        assert torch.equal(p, q)
