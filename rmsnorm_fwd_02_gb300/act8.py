"""Torch-facing API of activations kept in 8 bits between a training step's forward and backward:
allocates outputs and workspace with torch, then calls the C ABI (include/act8_train.h, which
defines the format).

    packed            = act8_pack(x)
    x                 = act8_unpack(packed, H, dtype=torch.bfloat16)

    y, rstd, x8       = rmsnorm_act8_fwd(x, w, eps)
    y, rstd, h8, h    = rmsnorm_act8_fwd(x_in, w, eps, residual=res)  # fused residual add
    dx, dw            = rmsnorm_act8_bwd(dy, x8, rstd, w, dh=None)
    y                 = rmsnorm_act8_train(x, w, eps)                 # autograd, keeps x8 and rstd
    y, h              = rmsnorm_act8_train(x_in, w, eps, residual=res)

Blocks of 32 values of the last axis share a power of two; a value is held within 1/127 of its
block's greatest magnitude (half that on average), in a byte, and a row of H values in
act8_row_bytes(H) = H + H/32 bytes, each padded to 16.  A block that holds an infinity or a NaN is
NaN.  Packed tensors are uint8 [..., act8_row_bytes(H)], contiguous.

act8_pack / act8_unpack: CUDA bfloat16, float16 or float32 tensors [..., H] of any H; the rows may
be strided where the leading axes merge into one, the last axis is contiguous.
rmsnorm_act8_*: the pair that rmsnorm_fwd / rmsnorm_bwd are, with the input that the backward
reads in 8 bits: rmsnorm_bwd's formulas at the held values (dw's additions carry their errors
from a thread's sums on, not throughout: act8_train.h).  It saves memory: a step takes longer than
rmsnorm_fwd and rmsnorm_bwd's.  x is bfloat16 or float16 [..., H],
H a multiple of 8 up to 8192, rows as above and at 16-byte boundaries; w is bfloat16, float16 or
float32 [H].  y, h, dx are contiguous; rstd is float32 [...]; dw float32 [H].  All results are
bit-reproducible.
"""
from __future__ import annotations

import functools
import math

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .dropout import _empty_strided, _flat, _layout, _like, _same_device
from .ops import EPS

_CODES = {torch.bfloat16: N.ACT8_BF16, torch.float32: N.ACT8_FP32, torch.float16: N.ACT8_FP16}
_NARROW = {torch.bfloat16: N.ACT8_BF16, torch.float16: N.ACT8_FP16}

# A call's checks, allocations and marshalling take longer than a small call's kernels, so the
# paths below ask each tensor once for what they need.  The current device comes without torch's
# lazy initialization (a CUDA tensor is there), where this torch has that (a private name).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(x: torch.Tensor):
    """A context for x's device where it is not the current one (the C ABI works on that), or
    None."""
    return None if x.get_device() == _current_device() else torch.cuda.device(x.device)


@functools.lru_cache(maxsize=4096)
def act8_row_bytes(H: int) -> int:
    """Bytes of a packed row of H values."""
    if H < 1:
        raise ValueError("a row has at least one value")
    return (H + 15) // 16 * 16 + ((H + 31) // 32 + 15) // 16 * 16


@functools.lru_cache(maxsize=4096)
def _layouts(shape):
    """Layouts (shape and strides) of tensors of this shape, of its rows' scalars, and of its packed
    rows."""
    return _layout(shape), _layout(shape[:-1]), _layout((*shape[:-1], act8_row_bytes(shape[-1])))


_width = functools.lru_cache(maxsize=4096)(lambda h: _layout((h,)))


def _rows(x: torch.Tensor, name: str):
    """x [..., H] as rows: their number, H and the elements between two."""
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name} must be [..., H]")
    h = shape[-1]
    rows = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    if x.is_contiguous() or rows == 0:
        return rows, h, h
    if h > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    try:
        v = x.view(rows, h)
    except RuntimeError:
        raise ValueError(f"{name}'s leading axes must merge into one") from None
    stride = v.stride(0) if rows > 1 else h
    if stride < h:
        raise ValueError(f"{name}'s rows must not overlap")
    return rows, h, stride


def _narrow(x: torch.Tensor, name: str) -> int:
    code = _NARROW.get(x.dtype)
    if code is None or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 or float16 tensor")
    return code


def _row_input(x: torch.Tensor, name: str):
    """_rows of a tensor whose rows the kernels copy in 16-byte pieces."""
    rows, h, stride = _rows(x, name)
    if h & 7 or h > 8192:
        raise ValueError(f"{name}'s last axis must be a multiple of 8 up to 8192")
    if stride & 7 or x.data_ptr() & 15:
        raise ValueError(f"{name}'s rows must start at 16-byte boundaries")
    return rows, h, stride


def _grad_rows(g: torch.Tensor, name: str):
    """Rows and H of a gradient (of any strides)."""
    shape = g.shape
    h = shape[-1] if len(shape) else 0
    if h < 8 or h & 7 or h > 8192:
        raise ValueError(f"{name}'s last axis must be a multiple of 8 up to 8192")
    return (shape[0] if len(shape) == 2 else math.prod(shape[:-1])), h


def _weight(w, h: int, name: str) -> int:
    code = _CODES.get(w.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    if w.dim() != 1 or w.numel() != h:
        raise ValueError(f"{name} must have shape ({h},)")
    return code


def _ready(t):
    """t, or a copy, contiguous at a 16-byte boundary; None stays."""
    return t if t is None or (t.is_contiguous() and not t.data_ptr() & 15) else _flat(t)


def _row_scalars(t, lead, name: str):
    if t.shape != lead or t.dtype != torch.float32:
        raise ValueError(f"{name} must have shape {tuple(lead)} and dtype float32")
    return t if t.is_contiguous() else t.contiguous()


def _packed(p, lead, h: int, name: str):
    """A packed tensor of rows [*lead, h], contiguous at a 16-byte boundary."""
    if p.dtype != torch.uint8 or p.shape != (*lead, act8_row_bytes(h)):
        raise ValueError(f"{name} must be a packed tensor: uint8 {(*lead, act8_row_bytes(h))}")
    return _ready(p)


def act8_pack(x):
    code = _CODES.get(x.dtype)
    if code is None or not x.is_cuda:
        raise TypeError("x must be a CUDA bfloat16, float16 or float32 tensor")
    rows, h, stride = _rows(x, "x")
    there = _elsewhere(x)
    if there is not None:
        with there:
            return act8_pack(x)
    packed = _empty_strided(*_layouts(x.shape)[2], torch.uint8)
    N.act8_train_pack(x, code, packed, rows, h, stride)
    return packed


def act8_unpack(packed, H, dtype=torch.bfloat16):
    if not packed.is_cuda:
        raise TypeError("packed must be a CUDA tensor")
    if dtype not in _CODES:
        raise TypeError("dtype must be bfloat16, float16 or float32")
    lead = packed.shape[:-1]
    packed = _packed(packed, lead, H, "packed")
    there = _elsewhere(packed)
    if there is not None:
        with there:
            return act8_unpack(packed, H, dtype)
    x = _empty_strided(*_layout((*lead, H)), dtype)
    N.act8_train_unpack(packed, x, _CODES[dtype], math.prod(lead), H)
    return x


def rmsnorm_act8_fwd(x, w, eps=EPS, residual=None):
    code = _narrow(x, "x")
    rows, h, s_x = _row_input(x, "x")
    w_code = _weight(w, h, "w")
    s_res = h
    if residual is not None:
        _like(x, "residual", residual)
        s_res = _row_input(residual, "residual")[2]
    _same_device(x, residual, w)
    there = _elsewhere(x)
    if there is not None:
        with there:
            return rmsnorm_act8_fwd(x, w, eps, residual)
    full, lead, kept = _layouts(x.shape)
    dtype = x.dtype
    y = _empty_strided(*full, dtype)
    h_out = _empty_strided(*full, dtype) if residual is not None else None
    rstd = _empty_strided(*lead, torch.float32)
    packed = _empty_strided(*kept, torch.uint8)
    N.rmsnorm_act8_train_fwd(x, residual, code, _ready(w), w_code, y, h_out, rstd, packed, rows, h,
                             s_x, s_res, float(eps))
    return (y, rstd, packed) if residual is None else (y, rstd, packed, h_out)


# a function of the shape alone
_bwd_bytes = functools.lru_cache(maxsize=4096)(
    lambda *shape: N.rmsnorm_act8_train_bwd_workspace_bytes(*shape))


def rmsnorm_act8_bwd(dy, x8, rstd, w, dh=None):
    code = _narrow(dy, "dy")
    rows, h = _grad_rows(dy, "dy")
    full, (lead, _), _ = _layouts(dy.shape)
    w_code = _weight(w, h, "w")
    x8 = _packed(x8, lead, h, "x8")
    rstd = _row_scalars(rstd, lead, "rstd")
    if dh is not None:
        _like(dy, "dh", dh)
    _same_device(dy, x8, rstd, w, dh)
    there = _elsewhere(dy)
    if there is not None:
        with there:
            return rmsnorm_act8_bwd(dy, x8, rstd, w, dh)
    dx = _empty_strided(*full, dy.dtype)
    dw = _empty_strided(*_width(h), torch.float32)
    nbytes = _bwd_bytes(rows, h)
    ws = _empty_strided((nbytes,), (1,), torch.uint8) if nbytes else None
    N.rmsnorm_act8_train_bwd(x8, _ready(dy), _ready(dh), code, rstd, _ready(w), w_code, dx, dw, ws,
                             nbytes, rows, h)
    return dx, dw


class RMSNormAct8Train(torch.autograd.Function):
    """Autograd wrapper: the forward keeps the normalized input in 8 bits, and rstd."""

    @staticmethod
    def forward(ctx, x, w, eps, residual):
        y, rstd, packed, *h = rmsnorm_act8_fwd(x, w, eps, residual)
        ctx.save_for_backward(packed, rstd, w)
        ctx.residual = residual is not None
        ctx.like = (x.shape, x.dtype)
        ctx.set_materialize_grads(False)
        return (y, *h) if ctx.residual else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        packed, rstd, w = ctx.saved_tensors
        if dy is None:
            if dh is None:
                return None, None, None, None
            dy = torch.zeros(ctx.like[0], dtype=ctx.like[1], device=packed.device)
        dx, dw = rmsnorm_act8_bwd(dy, packed, rstd, w, dh)
        return dx, dw.to(w.dtype), None, dx if ctx.residual else None


def rmsnorm_act8_train(x, w, eps=EPS, residual=None):
    return RMSNormAct8Train.apply(x, w, eps, residual)
