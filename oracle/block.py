"""FP64 oracle of a block's boundary (include/block_train.h) in numpy.  Shares no code with the
CUDA library.  Tensors are float64 [R, H], weights [H] or None, gate [N, H] or None."""
from __future__ import annotations

import numpy as np


def rstd(v, eps):
    return 1 / np.sqrt((v * v).mean(1) + eps)


def gate_rows(gate, rows, h):
    """The gate's factor of every row."""
    return np.ones((rows, h)) if gate is None else np.repeat(gate, rows // gate.shape[0], 0)


def fwd(x, residual, w_pre, w_post, gate, scale, residual_scale, eps):
    """y, h, rstd_pre, rstd_post; None where there is no such norm."""
    p = x
    r1 = r2 = y = None
    if w_post is not None:
        r1 = rstd(x, eps)
        p = x * r1[:, None] * w_post
    h = residual_scale * residual + scale * gate_rows(gate, *x.shape) * p
    if w_pre is not None:
        r2 = rstd(h, eps)
        y = h * r2[:, None] * w_pre
    return y, h, r2, r1


def norm_bwd(g, xhat, r):
    return r[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))


def bwd(dy, dh, x, h, r2, r1, w_pre, w_post, gate, scale, residual_scale):
    """Gradients of sum(dy * y) + sum(dh * h) at the given r's: dx, dresidual, dw_pre, dw_post,
    dgate, and t, the gradient of h."""
    dw_pre = dw_post = dgate = None
    if w_pre is not None:
        hhat = h * r2[:, None]
        t = norm_bwd(dy * w_pre, hhat, r2)
        dw_pre = (dy * hhat).sum(0)
        if dh is not None:
            t = t + dh
    else:
        t = dh
    g = gate_rows(gate, *t.shape)
    branch = scale * g * t
    p = x
    if w_post is not None:
        xhat = x * r1[:, None]
        p = xhat * w_post
        dw_post = (branch * xhat).sum(0)
        dx = norm_bwd(branch * w_post, xhat, r1)
    else:
        dx = branch
    if gate is not None:
        n, hh = gate.shape
        dgate = (scale * t * p).reshape(n, -1, hh).sum(1)
    return dx, residual_scale * t, dw_pre, dw_post, dgate, t
