"""Inputs, oracle calls and error bounds shared by the GPU tests of 8-bit activations and of a
block's boundary.

Bounds, from the roundings alone (U = 2^-24 FP32's, u the output type's half step):
  A row sum of H products takes at most 8 additions a thread, 2 within it, 5 in the warp and 16 of the
  warps' sums, so its error is within 32 U of the sum of magnitudes (and one rounding a product):
  SUM = 34 U.  rstd: half of that, the division, the eps, the root: 20 U relative.
  Each elementwise product or sum adds U of its magnitude; the factor scale * gate * w_post has
  two.  A column sum over a team's rows of n values: n + 8 additions (the last ones, over the
  teams, carry their errors along), each within U of the sum of magnitudes.
"""
import numpy as np
import torch

from oracle import act8 as OA
from oracle import block as OB
from rmsnorm_fwd_02_gb300 import _native as N

DEV = "cuda"
U = 2.0 ** -24
SUM = 34 * U
RSTD = 20 * U
EPS = float(np.float32(1e-6))


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def f32(v):
    return float(np.float32(v))


def check(got, want, err, what=""):
    """got within err of want, and then rounded to its type."""
    info = torch.finfo(got.dtype)
    got = f64(got)
    u, tiny = (0.0, 0.0) if info.bits == 32 else (info.eps / 2, info.smallest_normal * info.eps / 2)
    allow = err + u * (np.abs(want) + err) + tiny
    far = np.abs(got - want) / np.maximum(allow, 1e-300)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= allow).all(), (what, far.max(), np.argwhere(far > 1)[:4])


def check_fwd(out, x, residual, w_pre, w_post, gate, scale, residual_scale, eps=EPS, written=False):
    """rmsnorm_block_fwd's y, h, rstd_pre, rstd_post ([R, H] each) against the oracle."""
    y, h, rstd_pre, rstd_post = out
    a, b = f32(residual_scale), f32(scale)
    x, residual, w_pre, w_post, gate = (f64(t) for t in (x, residual, w_pre, w_post, gate))
    gate = None if gate is None else gate.reshape(-1, x.shape[1])
    ey, eh, er2, er1 = OB.fwd(x, residual, w_pre, w_post, gate, b, a, eps)
    branch = eh - a * residual
    dh = np.abs(branch) * (RSTD + 5 * U) + 2 * U * np.abs(a * residual) + U * np.abs(eh)
    check(h, eh, dh, "h")
    if w_post is not None:
        check(rstd_post, er1, RSTD * er1, "rstd_post")
    else:
        assert rstd_post is None
    if w_pre is None:
        assert y is None and rstd_pre is None
        return
    moved = RSTD + (np.abs(eh) * dh).sum(1) / np.maximum((eh * eh).sum(1), 1e-300)
    check(rstd_pre, er2, er2 * moved, "rstd_pre")
    check(y, ey, np.abs(ey) * (moved[:, None] + 3 * U) + dh * er2[:, None] * np.abs(w_pre), "y")


def team_rows(rows, h, n, packed):
    """Most rows that a team sums up in a row."""
    p = N.rmsnorm_block_train_launch_plan(rows, h, n, True, packed)
    return rows // (p["ctas"] * p["teams"]) + 1


def check_bwd(out, dy, dh, x, h, rstd_pre, rstd_post, w_pre, w_post, gate, scale, residual_scale):
    """rmsnorm_block_bwd's results against the oracle; x, h activations or packed rows."""
    a, b = f32(residual_scale), f32(scale)
    grad = dh if dy is None else dy
    rows, width = grad.shape
    packed = any(t is not None and t.dtype == torch.uint8 for t in (x, h))

    def value(t):
        if t is not None and t.dtype == torch.uint8:
            return OA.unpack(t.cpu().numpy(), width)
        return f64(t)

    x, h = value(x), value(h)
    dy, dh, r2, r1, w_pre, w_post, gate = (
        f64(t) for t in (dy, dh, rstd_pre, rstd_post, w_pre, w_post, gate))
    shape = None if gate is None else gate.shape
    gate = None if gate is None else gate.reshape(-1, width)
    n = 1 if gate is None else gate.shape[0]
    want = OB.bwd(dy, dh, x, h, r2, r1, w_pre, w_post, gate, b, a)
    t = want[5]
    et = np.zeros_like(t)
    chain = (team_rows(rows, width, n, packed) + 8) * U
    if w_pre is not None:
        g, hh = dy * w_pre, h * r2[:, None]
        c, mag = (g * hh).mean(1, keepdims=True), np.abs(g * hh).mean(1, keepdims=True)
        et = r2[:, None] * (4 * U * np.abs(g) + np.abs(hh) * (SUM * mag + 6 * U * np.abs(c)))
        et += 2 * U * (np.abs(t) + (0 if dh is None else np.abs(dh)))
        check(out[2], want[2], (2 * U + chain) * np.abs(dy * hh).sum(0), "dw_pre")
    else:
        assert out[2] is None
    check(out[1], want[1], abs(a) * (et + U * np.abs(t)), "dresidual")
    factor = b * OB.gate_rows(gate, rows, width) * (1 if w_post is None else w_post)
    m = factor * t
    em = np.abs(factor) * et + 3 * U * np.abs(m)
    xh = x
    if w_post is not None:
        xh = x * r1[:, None]
        c, mag = (m * xh).mean(1, keepdims=True), np.abs(m * xh).mean(1, keepdims=True)
        ec = SUM * mag + (em * np.abs(xh)).mean(1, keepdims=True) + 6 * U * np.abs(c)
        check(out[0], want[0], r1[:, None] * (em + 3 * U * np.abs(m) + np.abs(xh) * ec), "dx")
    else:
        check(out[0], want[0], em, "dx")
    if gate is None and w_post is None:
        assert out[3] is None and out[4] is None
        return
    # S, a sum for each sample
    by = lambda v: v.reshape(n, -1, width).sum(1)  # noqa: E731
    es = by(et * np.abs(xh)) + (2 * U + chain) * by(np.abs(t * xh))
    s = np.abs(by(t * xh))
    one = 1 if w_post is None else np.abs(w_post)
    if gate is not None:
        check(out[4], want[4].reshape(shape), (abs(b) * one * (es + 3 * U * s)).reshape(shape), "dgate")
    else:
        assert out[4] is None
    if w_post is not None:
        g = np.ones((1, width)) if gate is None else np.abs(gate)
        check(out[3], want[3], abs(b) * (g * (es + 4 * U * s)).sum(0), "dw_post")
    else:
        assert out[3] is None
