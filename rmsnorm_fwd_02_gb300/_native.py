"""ctypes binding of ``librmsnorm_train.so`` with the C ABI's names (include/rmsnorm_train.h,
include/layernorm_train.h, include/dropout_train.h, include/groupnorm_train.h,
include/act8_train.h and include/block_train.h).

Argument marshalling only: tensors become device pointers, the current torch stream
becomes the ``cudaStream_t``, sizes and strides are passed through, and a nonzero status
becomes an exception.  Every step of the computation runs in the CUDA library; there is
no fallback.  If the library is missing this module raises on first use.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librmsnorm_train.so")

RMSN_OK = 0
RMSN_W_BF16 = 0
RMSN_W_FP32 = 1

# every C entry point declared in include/rmsnorm_train.h, with its ctypes signature
_i64, _i32, _vp, _int, _f32, _size = (C.c_int64, C.c_int32, C.c_void_p, C.c_int, C.c_float,
                                      C.c_size_t)
_u64, _f64 = C.c_uint64, C.c_double
SIGNATURES = {
    "rmsnorm_train_fwd": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i32, _i32, _i64,
                                 _i64, _f32, _vp]),
    "rmsnorm_train_bwd_workspace_bytes": (_size, [_i64, _i32, _i32, _int]),
    "rmsnorm_train_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _size, _i64,
                                 _i32, _i32, _i64, _i64, _int, _vp]),
    "rmsnorm_train_bwd_noalloc": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _i64, _i32,
                                         _i32, _i64, _i64, _int, _vp]),
    "rmsnorm_train_bwd_recompute": (_int, [_vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _size,
                                           _i64, _i32, _i32, _i64, _i64, _f32, _int, _vp]),
    "rmsnorm_train_status_str": (C.c_char_p, [_int]),
    "rmsnorm_train_device_error": (_int, [C.POINTER(C.c_uint), _int]),
    "rmsnorm_train_launch_plan": (_int, [_i32, _int, C.POINTER(C.c_int64), _int]),
    # include/layernorm_train.h
    "layernorm_train_fwd": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i32, _f32, _vp]),
    "layernorm_train_bwd_workspace_bytes": (_size, [_i64, _i32, _int]),
    "layernorm_train_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp, _size,
                                   _i64, _i32, _int, _vp]),
    "layernorm_train_launch_plan": (_int, [_i32, _int, C.POINTER(C.c_int64), _int]),
    "layernorm_train_device_error": (_int, [C.POINTER(C.c_uint), _int]),
    # include/dropout_train.h
    "dropout_train_fwd": (_int, [_vp, _vp, _vp, _int, _i64, _f64, _u64, _u64, _vp, _vp]),
    "dropout_train_bwd": (_int, [_vp, _vp, _int, _i64, _f64, _u64, _u64, _vp, _vp]),
    "rmsnorm_dropout_train_fwd": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _vp, _i64, _i32, _i32,
                                         _i64, _i64, _f32, _f64, _u64, _u64, _vp, _vp]),
    "rmsnorm_dropout_train_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp,
                                         _size, _i64, _i32, _i32, _f64, _u64, _u64, _vp, _int,
                                         _vp]),
    # include/groupnorm_train.h
    "groupnorm_train_fwd_workspace_bytes": (_size, [_int, _i64, _i64, _i32, _i32]),
    "groupnorm_train_bwd_workspace_bytes": (_size, [_int, _i64, _i64, _i32, _i32]),
    "groupnorm_train_fwd": (_int, [_vp, _int, _vp, _vp, _int, _vp, _vp, _vp, _vp, _size, _i64,
                                   _i64, _i32, _i32, _i64, _i64, _f32, _int, _vp]),
    "groupnorm_train_bwd": (_int, [_vp, _vp, _int, _vp, _vp, _vp, _vp, _int, _vp, _vp, _vp, _vp,
                                   _size, _i64, _i64, _i32, _i32, _i64, _i64, _int, _vp]),
    "groupnorm_train_launch_plan": (_int, [_int, _i64, _i64, _i32, _i32, _int,
                                           C.POINTER(C.c_int64), _int]),
    # include/act8_train.h
    "act8_train_row_bytes": (_i64, [_i64]),
    "act8_train_pack": (_int, [_vp, _int, _vp, _i64, _i64, _i64, _vp]),
    "act8_train_unpack": (_int, [_vp, _vp, _int, _i64, _i64, _vp]),
    "rmsnorm_act8_train_fwd": (_int, [_vp, _vp, _int, _vp, _int, _vp, _vp, _vp, _vp, _i64, _i32,
                                      _i64, _i64, _f32, _vp]),
    "rmsnorm_act8_train_bwd_workspace_bytes": (_size, [_i64, _i32]),
    "rmsnorm_act8_train_bwd": (_int, [_vp, _vp, _vp, _int, _vp, _vp, _int, _vp, _vp, _vp, _size,
                                      _i64, _i32, _vp]),
    # include/block_train.h
    "rmsnorm_block_train_fwd": (_int, [_vp, _vp, _int, _vp, _vp, _int, _vp, _int, _i64, _vp, _vp,
                                       _vp, _vp, _vp, _vp, _i64, _i32, _i64, _i64, _f32, _f32,
                                       _f32, _vp]),
    "rmsnorm_block_train_bwd_workspace_bytes": (_size, [_i64, _i32, _i64]),
    "rmsnorm_block_train_bwd": (_int, [_vp, _vp, _vp, _vp, _int, _int, _vp, _vp, _vp, _vp, _int,
                                       _vp, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _size, _i64,
                                       _i32, _i64, _f32, _f32, _vp]),
    "rmsnorm_block_train_launch_plan": (_int, [_i64, _i32, _i64, _int, _int, C.POINTER(C.c_int64),
                                               _int]),
    "rmsnorm_block_train_device_error": (_int, [C.POINTER(C.c_uint), _int]),
}

DROPOUT_BF16, DROPOUT_FP32, DROPOUT_FP16 = 0, 1, 2
GROUPNORM_BF16, GROUPNORM_FP32, GROUPNORM_FP16 = 0, 1, 2
GROUPNORM_ACT_NONE, GROUPNORM_ACT_SILU, GROUPNORM_ACT_GELU = 0, 1, 2
GROUPNORM_PLAN_FIELDS = ("on_chip", "channels", "threads", "cluster_ctas", "ctas", "smem",
                         "units", "chunks")
ACT8_BF16, ACT8_FP32, ACT8_FP16 = 0, 1, 2
BLOCK_PLAN_FIELDS = ("vectors", "row_threads", "teams", "rows", "stages", "threads", "ctas", "smem")
BLOCK_PLAN_NO_NORM_BEHIND, BLOCK_PLAN_NO_NORM_BEFORE, BLOCK_PLAN_NO_GATE = 2, 4, 8
BLOCK_PLAN_ONE_INPUT, BLOCK_PLAN_ACT8_NORM = 16, 32

PLAN_FWD, PLAN_FWD_RESIDUAL, PLAN_BWD, PLAN_BWD_DH, PLAN_BWD_ND, PLAN_BWD_ND_DH = 0, 1, 2, 3, 4, 5
LN_PLAN_FWD, LN_PLAN_BWD = 0, 1
PLAN_FIELDS = ("vpt", "group_threads", "groups", "stages", "threads", "smem", "cls",
               "class_max_threads", "class_blocks_per_sm")
LN_PLAN_FIELDS = PLAN_FIELDS + ("cluster_ctas",)

_lib = None


class RmsnError(RuntimeError):
    """A nonzero status from the CUDA library."""

    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_str(status)})")
        self.status = status


def lib():
    """The loaded library.  Raises if it has not been built: there is no CPU path."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"CUDA library {LIB_PATH} is missing; build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_str(status: int) -> str:
    return lib().rmsnorm_train_status_str(status).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _raw_stream_object(device):
    return torch.cuda.current_stream(device).cuda_stream


# the current stream's handle alone, without a Stream object around it (2.5 us a call), where
# this torch has that (a private name)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream_object)


def _stream(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def rmsnorm_train_fwd(x, residual, w, w_dtype, y, h_out, rstd, T, nh, H, s_tok, s_head,
                      eps, stream=None):
    st = lib().rmsnorm_train_fwd(_ptr(x), _ptr(residual), _ptr(w), w_dtype, _ptr(y),
                                 _ptr(h_out), _ptr(rstd), T, nh, H, s_tok, s_head, eps,
                                 _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_fwd", st)


def rmsnorm_train_bwd_workspace_bytes(T, nh, H, deterministic):
    return int(lib().rmsnorm_train_bwd_workspace_bytes(T, nh, H, int(deterministic)))


def rmsnorm_train_bwd(x, dy, dh, rstd, w, w_dtype, dx, dw, workspace, workspace_bytes, T, nh,
                      H, s_tok, s_head, deterministic, stream=None):
    st = lib().rmsnorm_train_bwd(_ptr(x), _ptr(dy), _ptr(dh), _ptr(rstd), _ptr(w), w_dtype,
                                 _ptr(dx), _ptr(dw), _ptr(workspace), workspace_bytes, T, nh,
                                 H, s_tok, s_head, int(deterministic), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_bwd", st)


def rmsnorm_train_bwd_recompute(x, dy, dh, w, w_dtype, dx, dw, rstd_out, workspace,
                                workspace_bytes, T, nh, H, s_tok, s_head, eps, deterministic,
                                stream=None):
    st = lib().rmsnorm_train_bwd_recompute(_ptr(x), _ptr(dy), _ptr(dh), _ptr(w), w_dtype,
                                           _ptr(dx), _ptr(dw), _ptr(rstd_out), _ptr(workspace),
                                           workspace_bytes, T, nh, H, s_tok, s_head, eps,
                                           int(deterministic), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_bwd_recompute", st)


def rmsnorm_train_bwd_noalloc(x, dy, dh, rstd, w, w_dtype, dx, dw, T, nh, H, s_tok, s_head,
                              deterministic, stream=None):
    st = lib().rmsnorm_train_bwd_noalloc(_ptr(x), _ptr(dy), _ptr(dh), _ptr(rstd), _ptr(w),
                                         w_dtype, _ptr(dx), _ptr(dw), T, nh, H, s_tok, s_head,
                                         int(deterministic), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_bwd_noalloc", st)


def rmsnorm_train_status_str(status):
    return status_str(status)


def rmsnorm_train_device_error(reset=True):
    flags = C.c_uint(0)
    st = lib().rmsnorm_train_device_error(C.byref(flags), int(reset))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_device_error", st)
    return int(flags.value)


def rmsnorm_train_launch_plan(H, op):
    """The library's launch plan for one op (PLAN_*) at width H, as a dict."""
    out = (C.c_int64 * len(PLAN_FIELDS))()
    st = lib().rmsnorm_train_launch_plan(H, op, out, len(PLAN_FIELDS))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_train_launch_plan", st)
    return dict(zip(PLAN_FIELDS, (int(v) for v in out)))


# ---- LayerNorm (include/layernorm_train.h) ----------------------------------------------

def layernorm_train_fwd(x, w, b, wb_dtype, y, mean, rstd, R, H, eps, stream=None):
    st = lib().layernorm_train_fwd(_ptr(x), _ptr(w), _ptr(b), wb_dtype, _ptr(y), _ptr(mean),
                                   _ptr(rstd), R, H, eps, _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("layernorm_train_fwd", st)


def layernorm_train_bwd_workspace_bytes(R, H, deterministic):
    return int(lib().layernorm_train_bwd_workspace_bytes(R, H, int(deterministic)))


def layernorm_train_bwd(x, dy, mean, rstd, w, wb_dtype, dx, dw, db, workspace, workspace_bytes,
                        R, H, deterministic, stream=None):
    st = lib().layernorm_train_bwd(_ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(w), wb_dtype,
                                   _ptr(dx), _ptr(dw), _ptr(db), _ptr(workspace),
                                   workspace_bytes, R, H, int(deterministic), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("layernorm_train_bwd", st)


def layernorm_train_launch_plan(H, op):
    """The library's LayerNorm launch plan for op LN_PLAN_FWD / LN_PLAN_BWD, as a dict."""
    out = (C.c_int64 * len(LN_PLAN_FIELDS))()
    st = lib().layernorm_train_launch_plan(H, op, out, len(LN_PLAN_FIELDS))
    if st != RMSN_OK:
        raise RmsnError("layernorm_train_launch_plan", st)
    return dict(zip(LN_PLAN_FIELDS, (int(v) for v in out)))


def layernorm_train_device_error(reset=True):
    flags = C.c_uint(0)
    st = lib().layernorm_train_device_error(C.byref(flags), int(reset))
    if st != RMSN_OK:
        raise RmsnError("layernorm_train_device_error", st)
    return int(flags.value)


# ---- dropout (include/dropout_train.h) --------------------------------------------------

def dropout_train_fwd(x, residual, y, dtype, n, p, seed, offset, step, stream=None):
    st = lib().dropout_train_fwd(_ptr(x), _ptr(residual), _ptr(y), dtype, n, p, seed, offset,
                                 _ptr(step), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("dropout_train_fwd", st)


def dropout_train_bwd(dy, dx, dtype, n, p, seed, offset, step, stream=None):
    st = lib().dropout_train_bwd(_ptr(dy), _ptr(dx), dtype, n, p, seed, offset, _ptr(step),
                                 _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("dropout_train_bwd", st)


def rmsnorm_dropout_train_fwd(x, residual, w, w_dtype, y, h_out, rstd, T, nh, H, s_tok, s_head,
                              eps, p, seed, offset, step, stream=None):
    st = lib().rmsnorm_dropout_train_fwd(_ptr(x), _ptr(residual), _ptr(w), w_dtype, _ptr(y),
                                         _ptr(h_out), _ptr(rstd), T, nh, H, s_tok, s_head, eps,
                                         p, seed, offset, _ptr(step), _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_dropout_train_fwd", st)


def rmsnorm_dropout_train_bwd(h, dy, dh, rstd, w, w_dtype, dx, dresidual, dw, workspace,
                              workspace_bytes, T, nh, H, p, seed, offset, step, deterministic,
                              stream=None):
    st = lib().rmsnorm_dropout_train_bwd(_ptr(h), _ptr(dy), _ptr(dh), _ptr(rstd), _ptr(w),
                                         w_dtype, _ptr(dx), _ptr(dresidual), _ptr(dw),
                                         _ptr(workspace), workspace_bytes, T, nh, H, p, seed,
                                         offset, _ptr(step), int(deterministic),
                                         _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_dropout_train_bwd", st)


# ---- group norm (include/groupnorm_train.h) ---------------------------------------------

def groupnorm_train_fwd_workspace_bytes(dtype, N, S, C_, G):
    return int(lib().groupnorm_train_fwd_workspace_bytes(dtype, N, S, C_, G))


def groupnorm_train_bwd_workspace_bytes(dtype, N, S, C_, G):
    return int(lib().groupnorm_train_bwd_workspace_bytes(dtype, N, S, C_, G))


def groupnorm_train_fwd(x, dtype, w, b, wb_dtype, y, mean, rstd, workspace, workspace_bytes, N, S,
                        C_, G, s_n, s_s, eps, act, stream=None):
    st = lib().groupnorm_train_fwd(_ptr(x), dtype, _ptr(w), _ptr(b), wb_dtype, _ptr(y),
                                   _ptr(mean), _ptr(rstd), _ptr(workspace), workspace_bytes, N,
                                   S, C_, G, s_n, s_s, eps, act, _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("groupnorm_train_fwd", st)


def groupnorm_train_bwd(x, dy, dtype, mean, rstd, w, b, wb_dtype, dx, dw, db, workspace,
                        workspace_bytes, N, S, C_, G, s_n, s_s, act, stream=None):
    st = lib().groupnorm_train_bwd(_ptr(x), _ptr(dy), dtype, _ptr(mean), _ptr(rstd), _ptr(w),
                                   _ptr(b), wb_dtype, _ptr(dx), _ptr(dw), _ptr(db),
                                   _ptr(workspace), workspace_bytes, N, S, C_, G, s_n, s_s, act,
                                   _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("groupnorm_train_bwd", st)


def groupnorm_train_launch_plan(dtype, N, S, C_, G, backward):
    """The library's group norm launch plan for a shape, as a dict."""
    out = (C.c_int64 * len(GROUPNORM_PLAN_FIELDS))()
    st = lib().groupnorm_train_launch_plan(dtype, N, S, C_, G, int(backward), out,
                                           len(GROUPNORM_PLAN_FIELDS))
    if st != RMSN_OK:
        raise RmsnError("groupnorm_train_launch_plan", st)
    return dict(zip(GROUPNORM_PLAN_FIELDS, (int(v) for v in out)))


# ---- activations in 8 bits (include/act8_train.h) ---------------------------------------
#
# (Tensors that every call has give their pointers here directly: _ptr's tests are a tenth of a
# microsecond each, and these calls have up to twenty.)

def _opt(t):
    return None if t is None else t.data_ptr()


def act8_train_row_bytes(H):
    return int(lib().act8_train_row_bytes(H))


def act8_train_pack(x, dtype, packed, R, H, s_row, stream=None):
    st = lib().act8_train_pack(x.data_ptr(), dtype, packed.data_ptr(), R, H, s_row,
                               _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("act8_train_pack", st)


def act8_train_unpack(packed, y, dtype, R, H, stream=None):
    st = lib().act8_train_unpack(packed.data_ptr(), y.data_ptr(), dtype, R, H, _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("act8_train_unpack", st)


def rmsnorm_act8_train_fwd(x, residual, dtype, w, w_dtype, y, h_out, rstd, packed, R, H, s_x, s_res,
                           eps, stream=None):
    st = lib().rmsnorm_act8_train_fwd(x.data_ptr(), _opt(residual), dtype, w.data_ptr(), w_dtype,
                                      y.data_ptr(), _opt(h_out), rstd.data_ptr(),
                                      packed.data_ptr(), R, H, s_x, s_res, eps, _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_act8_train_fwd", st)


def rmsnorm_act8_train_bwd_workspace_bytes(R, H):
    return int(lib().rmsnorm_act8_train_bwd_workspace_bytes(R, H))


def rmsnorm_act8_train_bwd(packed, dy, dh, dtype, rstd, w, w_dtype, dx, dw, workspace,
                           workspace_bytes, R, H, stream=None):
    st = lib().rmsnorm_act8_train_bwd(packed.data_ptr(), dy.data_ptr(), _opt(dh), dtype,
                                      rstd.data_ptr(), w.data_ptr(), w_dtype, dx.data_ptr(),
                                      dw.data_ptr(), _opt(workspace), workspace_bytes, R, H,
                                      _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_act8_train_bwd", st)


# ---- a block's boundary (include/block_train.h) -----------------------------------------

def rmsnorm_block_train_fwd(x, residual, dtype, w_pre, w_post, w_dtype, gate, gate_dtype, N, y, h,
                            rstd_pre, rstd_post, x8, h8, R, H, s_x, s_res, scale, residual_scale,
                            eps, stream=None):
    st = lib().rmsnorm_block_train_fwd(x.data_ptr(), residual.data_ptr(), dtype, _opt(w_pre),
                                       _opt(w_post), w_dtype, _opt(gate), gate_dtype, N, _opt(y),
                                       h.data_ptr(), _opt(rstd_pre), _opt(rstd_post), _opt(x8),
                                       _opt(h8), R, H, s_x, s_res, scale, residual_scale, eps,
                                       _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_block_train_fwd", st)


def rmsnorm_block_train_bwd_workspace_bytes(R, H, N):
    return int(lib().rmsnorm_block_train_bwd_workspace_bytes(R, H, N))


def rmsnorm_block_train_bwd(dy, dh, x, h, packed, dtype, rstd_pre, rstd_post, w_pre, w_post,
                            w_dtype, gate, gate_dtype, N, dx, dresidual, dw_pre, dw_post, dgate,
                            workspace, workspace_bytes, R, H, s_x, scale, residual_scale,
                            stream=None):
    st = lib().rmsnorm_block_train_bwd(_opt(dy), _opt(dh), _opt(x), _opt(h), int(packed), dtype,
                                       _opt(rstd_pre), _opt(rstd_post), _opt(w_pre),
                                       _opt(w_post), w_dtype, _opt(gate), gate_dtype, N,
                                       dx.data_ptr(), dresidual.data_ptr(), _opt(dw_pre),
                                       _opt(dw_post), _opt(dgate), _opt(workspace),
                                       workspace_bytes, R, H, s_x, scale, residual_scale,
                                       _stream(stream))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_block_train_bwd", st)


def rmsnorm_block_train_launch_plan(R, H, N, backward, packed, form=0):
    """The library's launch plan of a block's boundary (both norms, a gate, dh), or of what the
    BLOCK_PLAN_* flags of `form` make of it, for a shape, as a dict."""
    out = (C.c_int64 * len(BLOCK_PLAN_FIELDS))()
    st = lib().rmsnorm_block_train_launch_plan(R, H, N, int(backward) | form, int(packed), out,
                                               len(BLOCK_PLAN_FIELDS))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_block_train_launch_plan", st)
    return dict(zip(BLOCK_PLAN_FIELDS, (int(v) for v in out)))


def rmsnorm_block_train_device_error(reset=True):
    flags = C.c_uint(0)
    st = lib().rmsnorm_block_train_device_error(C.byref(flags), int(reset))
    if st != RMSN_OK:
        raise RmsnError("rmsnorm_block_train_device_error", st)
    return int(flags.value)
