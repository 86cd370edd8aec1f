"""FP64 oracle of the group norm entry points (include/groupnorm_train.h), in torch's float64
on the device of its inputs: the textbook definition, two-pass variance, each activation and
its slope written out.  Shares no code with the CUDA library."""
from __future__ import annotations

import math

import torch


def act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return z


def slope(z, kind):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if kind == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(
            2 * math.pi)
    return torch.ones_like(z)


def stats(x, groups, eps):
    """x [N, S, C] float64: mean, rstd [N, G]."""
    n, s, c = x.shape
    v = x.view(n, s, groups, c // groups)
    mean = v.mean((1, 3))
    var = (v - mean[:, None, :, None]).square().mean((1, 3))
    return mean, 1 / torch.sqrt(var + eps)


def wide(t, c):
    """[N, G] -> [N, 1, C]"""
    return t.repeat_interleave(c // t.shape[1], dim=1)[:, None]


def fwd(x, w, b, groups, eps, kind):
    mean, rstd = stats(x, groups, eps)
    z = (x - wide(mean, x.shape[2])) * wide(rstd, x.shape[2]) * w + b
    return act(z, kind), mean, rstd


def group_mean(t, groups):
    """[N, S, C] -> its group means, [N, 1, C]"""
    n, s, c = t.shape
    return wide(t.view(n, s, groups, c // groups).mean((1, 3)), c)


def bwd(dy, x, mean, rstd, w, b, groups, kind):
    c = x.shape[2]
    xhat = (x - wide(mean, c)) * wide(rstd, c)
    dz = dy * slope(xhat * w + b, kind)
    g = dz * w
    dx = wide(rstd, c) * (g - group_mean(g, groups) - xhat * group_mean(g * xhat, groups))
    return dx, (dz * xhat).sum((0, 1)), dz.sum((0, 1))
