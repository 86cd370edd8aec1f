"""Torch-facing group norm API, channels last, with an activation behind the norm: allocates
outputs and workspace with torch, then calls the C ABI (include/groupnorm_train.h).

    y, mean, rstd  = groupnorm_fwd(x, w, b, groups, eps, act="none")
    dx, dw, db     = groupnorm_bwd(dy, x, mean, rstd, w, b, groups, act="none")
    y              = groupnorm_train(x, w, b, groups, eps, act)          # autograd

x is a CUDA bfloat16, float16 or float32 tensor [N, ..., C] with the channels last (an
[N, C, H, W] tensor in torch's channels_last format is x.permute(0, 2, 3, 1) here); N and the
merged places between may be strided, in whole 16-byte steps from a 16-byte boundary on.  C is
a multiple of 8 and of groups, up to 4096.  w and b are both bfloat16, float16 or float32 [C].
act is "none", "silu" or "gelu" (the exact form).  y, dx have x's shape and dtype and are
contiguous; mean and rstd are float32 [N, groups]; dw, db float32 [C].  All results are
bit-reproducible.
"""
from __future__ import annotations

import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .dropout import _DTYPES, _activation, _empty, _flat, _like, _on, _same_device

EPS = 1e-5

_ACTS = {"none": N.GROUPNORM_ACT_NONE, "silu": N.GROUPNORM_ACT_SILU, "gelu": N.GROUPNORM_ACT_GELU}


def _places(x: torch.Tensor, groups: int):
    dtype = _activation(x, "x")
    if x.dim() < 2:
        raise ValueError("x must be [N, ..., C]")
    shape = x.shape
    n, c = shape[0], shape[-1]
    s = shape[1] if len(shape) == 3 else math.prod(shape[1:-1])
    if n > 0 and s == 0:
        raise ValueError("x has samples without places")
    if groups < 1 or c % groups:
        raise ValueError(f"{c} channels do not divide into {groups} groups")
    if x.is_contiguous():
        return dtype, n, s, c, s * c, c
    if x.stride(-1) != 1 and c > 1:
        raise ValueError("the channels must be contiguous (channels last)")
    try:
        v = x.view(n, s, c)
    except RuntimeError:
        raise ValueError("the axes between samples and channels must merge into one") from None
    s_n = v.stride(0) if n > 1 else s * c
    s_s = v.stride(1) if s > 1 else c
    return dtype, n, s, c, s_n, s_s


def _params(x, w, b, c: int) -> int:
    if w.shape != (c,) or b.shape != (c,):
        raise ValueError(f"w and b must have shape ({c},)")
    if w.dtype != b.dtype or w.dtype not in _DTYPES:
        raise TypeError("w and b must both be bfloat16, float16 or float32")
    _same_device(x, w, b)
    return _DTYPES[w.dtype]


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}")
    return _ACTS[act]


# functions of the shape alone
_fwd_bytes = functools.lru_cache(maxsize=4096)(
    lambda *shape: N.groupnorm_train_fwd_workspace_bytes(*shape))
_bwd_bytes = functools.lru_cache(maxsize=4096)(
    lambda *shape: N.groupnorm_train_bwd_workspace_bytes(*shape))


def _workspace(nbytes: int):
    return _empty((nbytes,), torch.uint8) if nbytes else None


def groupnorm_fwd(x, w, b, groups, eps=EPS, act="none"):
    dtype, n, s, c, s_n, s_s = _places(x, groups)
    wb, code = _params(x, w, b, c), _act(act)
    with _on(x):
        y = _empty(x.shape, x.dtype)
        mean = _empty((n, groups), torch.float32)
        rstd = _empty((n, groups), torch.float32)
        nbytes = _fwd_bytes(dtype, n, s, c, groups)
        N.groupnorm_train_fwd(x, dtype, w.contiguous(), b.contiguous(), wb, y, mean, rstd,
                              _workspace(nbytes), nbytes, n, s, c, groups, s_n, s_s,
                              float(eps), code)
    return y, mean, rstd


def groupnorm_bwd(dy, x, mean, rstd, w, b, groups, act="none"):
    dtype, n, s, c, s_n, s_s = _places(x, groups)
    wb, code = _params(x, w, b, c), _act(act)
    _like(x, "dy", dy)
    for t in (mean, rstd):
        if t.shape != (n, groups) or t.dtype != torch.float32:
            raise ValueError(f"mean and rstd must have shape ({n}, {groups}) and dtype float32")
    _same_device(x, dy, mean, rstd)
    with _on(x):
        dx = _empty(x.shape, x.dtype)
        dw = _empty((c,), torch.float32)
        db = _empty((c,), torch.float32)
        nbytes = _bwd_bytes(dtype, n, s, c, groups)
        N.groupnorm_train_bwd(x, _flat(dy), dtype, mean.contiguous(), rstd.contiguous(),
                              w.contiguous(), b.contiguous(), wb, dx, dw, db,
                              _workspace(nbytes), nbytes, n, s, c, groups, s_n, s_s, code)
    return dx, dw, db


class GroupNormTrain(torch.autograd.Function):
    """Autograd wrapper: the forward keeps x, mean and rstd; the backward forms the
    activation's slope again."""

    @staticmethod
    def forward(ctx, x, w, b, groups, eps, act):
        y, mean, rstd = groupnorm_fwd(x, w, b, groups, eps, act)
        ctx.save_for_backward(x, mean, rstd, w, b)
        ctx.args = (groups, act)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, w, b = ctx.saved_tensors
        dx, dw, db = groupnorm_bwd(dy, x, mean, rstd, w, b, *ctx.args)
        return dx, dw.to(w.dtype), db.to(b.dtype), None, None, None


def groupnorm_train(x, w, b, groups, eps=EPS, act="none"):
    return GroupNormTrain.apply(x, w, b, groups, eps, act)
