"""Torch-facing API of a block's boundary: the norm behind a block, its gate, the residual add with
its scales, and the norm before the next block, in one pass each way.  Allocates outputs and
workspace with torch, then calls the C ABI (include/block_train.h).

    y, h, rstd_pre, rstd_post          = rmsnorm_block_fwd(x, residual, w_pre, w_post, gate,
                                                           scale, residual_scale, eps)
    y, h, rstd_pre, rstd_post, x8, h8  = rmsnorm_block_fwd(..., act8=True)
    dx, dresidual, dw_pre, dw_post, dgate = rmsnorm_block_bwd(dy, x, h, rstd_pre, rstd_post, w_pre,
                                                           w_post, gate, scale, residual_scale,
                                                           dh=None)
    y, h                               = rmsnorm_block_train(...)        # autograd

    h = residual_scale * residual + scale * gate * (rmsnorm(x) * w_post)
    y = rmsnorm(h) * w_pre                       (of h before it is rounded for writing)

x is the block's output, [..., H], CUDA bfloat16 or float16; residual has its shape and dtype.
Rows may be strided where the leading axes merge into one, at 16-byte boundaries; H is a
multiple of 8 up to 8192.  w_post and w_pre are [H], both bfloat16, float16 or float32; without
w_post the branch is x itself, without w_pre there is no y, and one of them is given.  gate is
None, [H], or [N, H] with a row for each of N equally long runs of rows (the samples of a batch
[N, ..., H]), of any of the three dtypes.  scale, residual_scale and eps are numbers, which get no
gradient.

What is not asked for is None in the results.  With act8 the forward also returns what its
backward reads of x and h in 8 bits (act8.py); rmsnorm_block_bwd takes either kind, x and h
alike: h with a norm before, x with a norm behind or a gate (else None is fine).  h, y and
gradients of activations are contiguous; rstd_* are float32 [...]; dw_* and dgate float32.  All
results are bit-reproducible.
"""
from __future__ import annotations

import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .act8 import (_CODES, _elsewhere, _grad_rows, _layouts, _narrow, _packed, _ready, _row_input,
                   _row_scalars, _weight, _width)
from .dropout import _empty_strided, _layout, _like, _same_device
from .ops import EPS


def _factors(rows: int, h: int, w_pre, w_post, gate, scale, residual_scale):
    """Checks the weights, the gate and the scales; the weights' and the gate's codes, N."""
    if w_pre is not None:
        code = _weight(w_pre, h, "w_pre")
        if w_post is not None and _weight(w_post, h, "w_post") != code:
            raise TypeError("w_pre and w_post must have one dtype")
    elif w_post is not None:
        code = _weight(w_post, h, "w_post")
    else:
        raise ValueError("one of w_pre and w_post must be given")
    gate_code, n = 0, 1
    if gate is not None:
        gate_code = _CODES.get(gate.dtype)
        if gate_code is None:
            raise TypeError("gate must be bfloat16, float16 or float32")
        shape = gate.shape
        if len(shape) not in (1, 2) or shape[-1] != h:
            raise ValueError(f"gate must be [{h}] or [N, {h}]")
        if len(shape) == 2:
            n = shape[0]
        if n < 1 or rows % n:
            raise ValueError(f"{rows} rows do not divide into gate's {n}")
    if not (math.isfinite(scale) and math.isfinite(residual_scale)):
        raise ValueError("scale and residual_scale must be finite")
    return code, gate_code, n


def rmsnorm_block_fwd(x, residual, w_pre=None, w_post=None, gate=None, scale=1.0,
                      residual_scale=1.0, eps=EPS, act8=False):
    code = _narrow(x, "x")
    rows, h, s_x = _row_input(x, "x")
    _like(x, "residual", residual)
    s_res = _row_input(residual, "residual")[2]
    w_code, gate_code, n = _factors(rows, h, w_pre, w_post, gate, scale, residual_scale)
    _same_device(x, residual, w_pre, w_post, gate)
    there = _elsewhere(x)
    if there is not None:
        with there:
            return rmsnorm_block_fwd(x, residual, w_pre, w_post, gate, scale, residual_scale, eps,
                                     act8)
    full, lead, kept = _layouts(x.shape)
    dtype = x.dtype
    out_h = _empty_strided(*full, dtype)
    y = rstd_pre = rstd_post = x8 = h8 = None
    if w_pre is not None:
        y = _empty_strided(*full, dtype)
        rstd_pre = _empty_strided(*lead, torch.float32)
    if w_post is not None:
        rstd_post = _empty_strided(*lead, torch.float32)
    if act8:
        if w_post is not None or gate is not None:
            x8 = _empty_strided(*kept, torch.uint8)
        if w_pre is not None:
            h8 = _empty_strided(*kept, torch.uint8)
    N.rmsnorm_block_train_fwd(x, residual, code, _ready(w_pre), _ready(w_post), w_code,
                              _ready(gate), gate_code, n, y, out_h, rstd_pre, rstd_post, x8, h8,
                              rows, h, s_x, s_res, float(scale), float(residual_scale),
                              float(eps))
    out = (y, out_h, rstd_pre, rstd_post)
    return out + (x8, h8) if act8 else out


# a function of the shape alone
_bwd_bytes = functools.lru_cache(maxsize=4096)(
    lambda *shape: N.rmsnorm_block_train_bwd_workspace_bytes(*shape))


def _kept(t, grad, lead, h: int, name: str):
    """A kept activation of grad's rows: (tensor, elements between rows, whether it is packed)."""
    if t is None:
        raise ValueError(f"{name} must be given")
    if t.dtype == torch.uint8:
        return _packed(t, lead, h, name), h, True
    _like(grad, name, t)
    return t, _row_input(t, name)[2], False


def rmsnorm_block_bwd(dy, x, h, rstd_pre, rstd_post, w_pre=None, w_post=None, gate=None, scale=1.0,
                      residual_scale=1.0, dh=None):
    if (dy is None) != (w_pre is None):
        raise ValueError("dy must be given with w_pre, and only then")
    grad, name = (dh, "dh") if dy is None else (dy, "dy")
    if grad is None:
        raise ValueError("dh must be given without w_pre")
    code = _narrow(grad, name)
    rows, width = _grad_rows(grad, name)
    full, (lead, _), _ = _layouts(grad.shape)
    if dh is not None and dy is not None:
        _like(dy, "dh", dh)
    w_code, gate_code, n = _factors(rows, width, w_pre, w_post, gate, scale, residual_scale)
    s_x, packed = width, None
    if w_pre is not None:
        h, s_h, packed = _kept(h, grad, lead, width, "h")
        if s_h != width:
            raise ValueError("h must be contiguous")
        rstd_pre = _row_scalars(rstd_pre, lead, "rstd_pre")
    else:
        h = rstd_pre = None
    if w_post is not None or gate is not None:
        x, s_x, x_packed = _kept(x, grad, lead, width, "x")
        if packed is not None and packed != x_packed:
            raise ValueError("x and h must both be activations or both packed")
        packed = x_packed
    else:
        x = None
    rstd_post = _row_scalars(rstd_post, lead, "rstd_post") if w_post is not None else None
    _same_device(grad, dy, dh, x, h, rstd_pre, rstd_post, w_pre, w_post, gate)
    there = _elsewhere(grad)
    if there is not None:
        with there:
            return rmsnorm_block_bwd(dy, x, h, rstd_pre, rstd_post, w_pre, w_post, gate, scale,
                                     residual_scale, dh)
    one = _width(width)
    dx = _empty_strided(*full, grad.dtype)
    dres = _empty_strided(*full, grad.dtype)
    dw_pre = _empty_strided(*one, torch.float32) if w_pre is not None else None
    dw_post = _empty_strided(*one, torch.float32) if w_post is not None else None
    dgate = _empty_strided(*_layout(gate.shape), torch.float32) if gate is not None else None
    nbytes = _bwd_bytes(rows, width, n)
    ws = _empty_strided((nbytes,), (1,), torch.uint8) if nbytes else None
    N.rmsnorm_block_train_bwd(_ready(dy), _ready(dh), x, h, packed, code, rstd_pre, rstd_post,
                              _ready(w_pre), _ready(w_post), w_code, _ready(gate), gate_code, n,
                              dx, dres, dw_pre, dw_post, dgate, ws, nbytes, rows, width, s_x,
                              float(scale), float(residual_scale))
    return dx, dres, dw_pre, dw_post, dgate


class RMSNormBlockTrain(torch.autograd.Function):
    """Autograd wrapper: the forward keeps x and h (each only where the backward reads it), in 8
    bits with act8, and the rows' rstd."""

    @staticmethod
    def forward(ctx, x, residual, w_pre, w_post, gate, scale, residual_scale, eps, act8):
        y, h, rstd_pre, rstd_post, *kept = rmsnorm_block_fwd(
            x, residual, w_pre, w_post, gate, scale, residual_scale, eps, act8)
        if not act8:
            kept = (x if w_post is not None or gate is not None else None,
                    h if w_pre is not None else None)
        ctx.save_for_backward(*kept, rstd_pre, rstd_post, w_pre, w_post, gate)
        ctx.scales = (scale, residual_scale)
        ctx.like = (x.shape, x.dtype, x.device)
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        kept_x, kept_h, rstd_pre, rstd_post, w_pre, w_post, gate = ctx.saved_tensors
        if dy is None and dh is None:
            return (None,) * 9
        if dy is None and w_pre is not None:
            dy = torch.zeros(ctx.like[0], dtype=ctx.like[1], device=ctx.like[2])
        grads = rmsnorm_block_bwd(dy, kept_x, kept_h, rstd_pre, rstd_post, w_pre, w_post, gate,
                                  *ctx.scales, dh=dh)
        grads = [g if p is None else g.to(p.dtype)
                 for g, p in zip(grads, (None, None, w_pre, w_post, gate))]
        return (*grads, None, None, None, None)


def _number(v, name: str) -> float:
    """A scale as the number it is now (a tensor could change before the backward)."""
    if isinstance(v, torch.Tensor) and v.requires_grad and torch.is_grad_enabled():
        raise TypeError(f"{name} is a number and gets no gradient (a gate does)")
    return float(v)


def rmsnorm_block_train(x, residual, w_pre=None, w_post=None, gate=None, scale=1.0,
                        residual_scale=1.0, eps=EPS, act8=False):
    return RMSNormBlockTrain.apply(x, residual, w_pre, w_post, gate, _number(scale, "scale"),
                                   _number(residual_scale, "residual_scale"), eps, act8)
