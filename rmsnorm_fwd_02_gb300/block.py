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
[N, ..., H]), of any of the three dtypes.

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
from .act8 import _CODES, _WIDTHS, _layouts, _narrow, _packed, _row_input, _row_scalars, _weight
from .dropout import _empty_strided, _flat, _layout, _like, _on, _same_device
from .ops import EPS


def _factors(x, others, rows: int, h: int, w_pre, w_post, gate, scale, residual_scale):
    """Checks the weights, the gate and the scales, and that all tensors are on x's device; the
    weights' and the gate's codes, N."""
    if w_pre is None and w_post is None:
        raise ValueError("one of w_pre and w_post must be given")
    codes = [_weight(w, h, name) for w, name in ((w_pre, "w_pre"), (w_post, "w_post"))
             if w is not None]
    if codes[0] != codes[-1]:
        raise TypeError("w_pre and w_post must have one dtype")
    gate_code, n = 0, 1
    if gate is not None:
        if gate.dtype not in _CODES:
            raise TypeError("gate must be bfloat16, float16 or float32")
        gate_code = _CODES[gate.dtype]
        if gate.dim() not in (1, 2) or gate.shape[-1] != h:
            raise ValueError(f"gate must be [{h}] or [N, {h}]")
        n = gate.shape[0] if gate.dim() == 2 else 1
        if n < 1 or rows % n:
            raise ValueError(f"{rows} rows do not divide into gate's {n}")
    _same_device(x, *others, w_pre, w_post, gate)
    if not (math.isfinite(scale) and math.isfinite(residual_scale)):
        raise ValueError("scale and residual_scale must be finite")
    return codes[0], gate_code, n


def _opt_flat(t):
    return None if t is None else _flat(t)


def rmsnorm_block_fwd(x, residual, w_pre=None, w_post=None, gate=None, scale=1.0,
                      residual_scale=1.0, eps=EPS, act8=False):
    code = _narrow(x, "x")
    rows, h, s_x = _row_input(x, "x")
    _like(x, "residual", residual)
    _, _, s_res = _row_input(residual, "residual")
    w_code, gate_code, n = _factors(x, (residual,), rows, h, w_pre, w_post, gate, scale, residual_scale)
    full, lead, kept = _layouts(x.shape)
    dtype = x.dtype
    with _on(x):
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
        N.rmsnorm_block_train_fwd(x, residual, code, _opt_flat(w_pre), _opt_flat(w_post), w_code,
                                  _opt_flat(gate), gate_code, n, y, out_h, rstd_pre, rstd_post,
                                  x8, h8, rows, h, s_x, s_res, float(scale),
                                  float(residual_scale), float(eps))
    out = (y, out_h, rstd_pre, rstd_post)
    return out + (x8, h8) if act8 else out


# a function of the shape alone
_bwd_bytes = functools.lru_cache(maxsize=4096)(
    lambda *shape: N.rmsnorm_block_train_bwd_workspace_bytes(*shape))


def _kept(t, grad, h: int, name: str):
    """A kept activation of grad's rows: (tensor, elements between rows, whether it is packed)."""
    if t is None:
        raise ValueError(f"{name} must be given")
    if t.dtype == torch.uint8:
        return _packed(t, grad.shape[:-1], h, name), h, True
    _like(grad, name, t)
    _, _, stride = _row_input(t, name)
    return t, stride, False


def rmsnorm_block_bwd(dy, x, h, rstd_pre, rstd_post, w_pre=None, w_post=None, gate=None, scale=1.0,
                      residual_scale=1.0, dh=None):
    if (dy is None) != (w_pre is None):
        raise ValueError("dy must be given with w_pre, and only then")
    grad = dh if dy is None else dy
    if grad is None:
        raise ValueError("dh must be given without w_pre")
    code = _narrow(grad, "dh" if dy is None else "dy")
    width = grad.shape[-1] if grad.dim() else 0
    if width < 8 or width % 8 or width > 8192:
        raise ValueError("the gradients' last axis must be a multiple of 8 up to 8192")
    rows = math.prod(grad.shape[:-1])
    if dh is not None:
        _like(grad, "dh", dh)
        dh = _flat(dh)
    dy = _opt_flat(dy)
    kinds, s_x = set(), width
    if w_pre is not None:
        h, s_h, packed = _kept(h, grad, width, "h")
        if not packed and s_h != width:
            raise ValueError("h must be contiguous")
        kinds.add(packed)
        rstd_pre = _row_scalars(rstd_pre, grad, "rstd_pre")
    else:
        h = rstd_pre = None
    if w_post is not None or gate is not None:
        x, s_x, packed = _kept(x, grad, width, "x")
        kinds.add(packed)
    else:
        x = None
    rstd_post = _row_scalars(rstd_post, grad, "rstd_post") if w_post is not None else None
    if len(kinds) > 1:
        raise ValueError("x and h must both be activations or both packed")
    w_code, gate_code, n = _factors(grad, (dy, dh, x, h, rstd_pre, rstd_post), rows, width, w_pre,
                                    w_post, gate, scale, residual_scale)
    with _on(grad):
        full, one = _layout(grad.shape), _WIDTHS(width)
        dx = _empty_strided(*full, grad.dtype)
        dres = _empty_strided(*full, grad.dtype)
        dw_pre = _empty_strided(*one, torch.float32) if w_pre is not None else None
        dw_post = _empty_strided(*one, torch.float32) if w_post is not None else None
        dgate = _empty_strided(*_layout(gate.shape), torch.float32) if gate is not None else None
        nbytes = _bwd_bytes(rows, width, n)
        ws = _empty_strided((nbytes,), (1,), torch.uint8) if nbytes else None
        N.rmsnorm_block_train_bwd(dy, dh, x, h, packed, code, rstd_pre, rstd_post,
                                  _opt_flat(w_pre), _opt_flat(w_post), w_code, _opt_flat(gate),
                                  gate_code, n, dx, dres, dw_pre, dw_post, dgate, ws, nbytes, rows,
                                  width, s_x, float(scale), float(residual_scale))
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


def rmsnorm_block_train(x, residual, w_pre=None, w_post=None, gate=None, scale=1.0,
                        residual_scale=1.0, eps=EPS, act8=False):
    return RMSNormBlockTrain.apply(x, residual, w_pre, w_post, gate, scale, residual_scale, eps,
                                   act8)
