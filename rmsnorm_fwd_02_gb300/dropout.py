"""Torch-facing dropout API: allocates outputs and workspace with torch, then calls the C ABI
(include/dropout_train.h, which defines the keep mask).

    y            = dropout_fwd(x, p, seed, offset=0, step=None, residual=None)
    dx           = dropout_bwd(dy, p, seed, offset=0, step=None)
    y            = dropout_train(x, p, seed, offset, step, residual)   # autograd

    y, rstd, h   = rmsnorm_dropout_fwd(x, residual, w, p, seed, offset=0, step=None, eps)
    dx, dres, dw = rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, offset=0, step=None,
                                       deterministic=True, dh=None)
    y, h         = rmsnorm_dropout_train(x, residual, w, p, seed, offset, step, eps)  # autograd

The second group is rmsnorm_fwd / rmsnorm_bwd's residual form with dropout on the added
branch: h = residual + dropout(x), y = rmsnorm(h) * w, in one pass each way.

The mask is a function of (seed, offset + step, p, element index) and is never stored: the
backward draws it again from the same values.  seed and offset are whole numbers in [0, 2^64);
step is None or a one-element int64 CUDA tensor that the kernels read when they run, so that a
captured graph draws new masks at each replay once the program has advanced it (after the
backward: autograd refuses a step changed in between).  Calls whose masks have to be
independent need different seeds, or different offset + step.

dropout_*: contiguous CUDA tensors of any shape, bfloat16, float16 or float32; residual has x's
shape and dtype.  rmsnorm_dropout_*: as rmsnorm_fwd with a residual; h is contiguous.  The
kernels read whole 16-byte vectors: an x that starts between two is refused, a gradient (or
dropout_fwd's residual) is copied first.  All tensors of a call are on one device.
"""
from __future__ import annotations

import contextlib
import functools

import torch
from torch.autograd.function import once_differentiable

from . import _native as N
from .ops import EPS, _view, _wdtype

_DTYPES = {torch.bfloat16: N.DROPOUT_BF16, torch.float32: N.DROPOUT_FP32,
           torch.float16: N.DROPOUT_FP16}


def _empty_strided_dispatched(shape, stride, dtype):
    return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")


# Outputs and workspaces, which the kernels write whole, come from torch's allocation of a CUDA
# tensor past the dispatcher, where this torch has it (a private name): through torch.empty, the
# allocations of a small call take longer than its launch (three of them and the launch 16 us,
# against 10).  Dispatch modes and torch's filling of uninitialized memory do not see them; the
# caching allocator, its pools and its streams are the same.
try:
    _empty_strided = torch._C._dynamo.guards._empty_strided_cuda
except AttributeError:
    _empty_strided = _empty_strided_dispatched


@functools.lru_cache(maxsize=4096)
def _layout(shape):
    """shape and its contiguous strides as plain tuples."""
    stride, n = [], 1
    for k in reversed(shape):
        stride.append(n)
        n *= k if k > 1 else 1
    return tuple(shape), tuple(reversed(stride))


def _empty(shape, dtype: torch.dtype) -> torch.Tensor:
    """An uninitialized contiguous tensor on the current device."""
    return _empty_strided(*_layout(shape), dtype)


_HERE = contextlib.nullcontext()


def _on(x: torch.Tensor):
    """A context in which x's device is the current one (the C ABI works on that)."""
    if x.get_device() == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(x.device)


def _same_device(x: torch.Tensor, *others):
    dev = x.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")


def _like(x: torch.Tensor, name: str, t):
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{name} must have shape {tuple(x.shape)} and dtype {x.dtype}")


def _flat(t):
    """t, or a copy, contiguous and at a 16-byte boundary: a gradient can be a slice of another
    tensor that starts anywhere."""
    t = t.contiguous()
    return t.clone(memory_format=torch.contiguous_format) if t.data_ptr() & 15 else t


def _generator(p, seed, offset, step, x):
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be between 0 and 1")
    for name, v in (("seed", seed), ("offset", offset)):
        if not isinstance(v, int) or not 0 <= v < 1 << 64:
            raise ValueError(f"{name} must be a whole number in [0, 2^64)")
    if step is not None:
        if step.dtype != torch.int64 or not step.is_cuda or step.numel() != 1:
            raise TypeError("step must be a one-element CUDA int64 tensor")
        _same_device(x, step)
    return p, seed, offset, step


def _activation(x: torch.Tensor, name: str) -> int:
    if x.dtype not in _DTYPES or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16, float16 or float32 tensor")
    return _DTYPES[x.dtype]


def dropout_fwd(x, p, seed, offset=0, step=None, residual=None):
    dtype = _activation(x, "x")
    gen = _generator(p, seed, offset, step, x)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None:
        _like(x, "residual", residual)
        _same_device(x, residual)
        residual = _flat(residual)
    with _on(x):
        y = _empty(x.shape, x.dtype)
        N.dropout_train_fwd(x, residual, y, dtype, x.numel(), *gen)
    return y


def dropout_bwd(dy, p, seed, offset=0, step=None):
    dtype = _activation(dy, "dy")
    gen = _generator(p, seed, offset, step, dy)
    dy = _flat(dy)
    with _on(dy):
        dx = _empty(dy.shape, dy.dtype)
        N.dropout_train_bwd(dy, dx, dtype, dy.numel(), *gen)
    return dx


class DropoutTrain(torch.autograd.Function):
    """Autograd wrapper: nothing but the generator's arguments is kept for the backward."""

    @staticmethod
    def forward(ctx, x, p, seed, offset, step, residual):
        ctx.args = (p, seed, offset)
        ctx.residual = residual is not None
        ctx.save_for_backward(*(() if step is None else (step,)))
        return dropout_fwd(x, p, seed, offset, step, residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        step = ctx.saved_tensors[0] if ctx.saved_tensors else None
        dx = dropout_bwd(dy, *ctx.args, step) if ctx.needs_input_grad[0] else None
        return dx, None, None, None, None, dy if ctx.residual else None


def dropout_train(x, p, seed, offset=0, step=None, residual=None):
    return DropoutTrain.apply(x, p, seed, offset, step, residual)


def rmsnorm_dropout_fwd(x, residual, w, p, seed, offset=0, step=None, eps=EPS):
    T, nh, H, s_tok, s_head = _view(x)
    gen = _generator(p, seed, offset, step, x)
    if residual.shape != x.shape or residual.stride() != x.stride() or residual.dtype != x.dtype:
        raise ValueError("residual must have x's shape, strides and dtype")
    if w.shape != (H,):
        raise ValueError(f"w must have shape ({H},)")
    _same_device(x, residual, w)
    w = w.contiguous()
    with _on(x):
        y = _empty(x.shape, torch.bfloat16)
        h = _empty(x.shape, torch.bfloat16)
        rstd = _empty(x.shape[:-1], torch.float32)
        N.rmsnorm_dropout_train_fwd(x, residual, w, _wdtype(w), y, h, rstd, T, nh, H, s_tok,
                                    s_head, float(eps), *gen)
    return y, rstd, h


def rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, offset=0, step=None, deterministic=True,
                        dh=None):
    T, nh, H, _, _ = _view(h)
    gen = _generator(p, seed, offset, step, h)
    if not h.is_contiguous():
        raise ValueError("h must be contiguous")
    _like(h, "dy", dy)
    if dh is not None:
        _like(h, "dh", dh)
        dh = _flat(dh)
    if rstd.shape != h.shape[:-1] or rstd.dtype != torch.float32:
        raise ValueError(f"rstd must have shape {tuple(h.shape[:-1])} and dtype float32")
    if w.shape != (H,):
        raise ValueError(f"w must have shape ({H},)")
    _same_device(h, dy, dh, rstd, w)
    dy = _flat(dy)
    w = w.contiguous()
    with _on(h):
        dx = _empty(h.shape, torch.bfloat16)
        dres = _empty(h.shape, torch.bfloat16)
        dw = _empty((H,), torch.float32)
        nbytes = N.rmsnorm_train_bwd_workspace_bytes(T, nh, H, deterministic)
        ws = _empty((nbytes,), torch.uint8) if nbytes else None
        N.rmsnorm_dropout_train_bwd(h, dy, dh, rstd.contiguous(), w, _wdtype(w), dx, dres, dw,
                                    ws, nbytes, T, nh, H, *gen, deterministic)
    return dx, dres, dw


class RMSNormDropoutTrain(torch.autograd.Function):
    """Autograd wrapper of the dropout form: the forward keeps h and rstd, no mask."""

    @staticmethod
    def forward(ctx, x, residual, w, p, seed, offset, step, eps, deterministic):
        ctx.args = (p, seed, offset)
        ctx.deterministic = deterministic
        ctx.has_step = step is not None
        y, rstd, h = rmsnorm_dropout_fwd(x, residual, w, p, seed, offset, step, eps)
        ctx.save_for_backward(h, rstd, w, *((step,) if ctx.has_step else ()))
        ctx.set_materialize_grads(False)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, rstd, w = ctx.saved_tensors[:3]
        step = ctx.saved_tensors[3] if ctx.has_step else None
        if dy is None:
            dy = torch.zeros_like(h)
        dx, dres, dw = rmsnorm_dropout_bwd(dy, h, rstd, w, *ctx.args, step, ctx.deterministic,
                                           dh)
        return dx, dres, dw.to(w.dtype), None, None, None, None, None, None


def rmsnorm_dropout_train(x, residual, w, p, seed, offset=0, step=None, eps=EPS,
                          deterministic=True):
    return RMSNormDropoutTrain.apply(x, residual, w, p, seed, offset, step, eps, deterministic)
