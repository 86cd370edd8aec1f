"""The dropout entry points of the C-ABI library without a GPU: declared, exported and bound;
bad arguments rejected before the first CUDA runtime call, in the C ABI and in the torch API."""
import ctypes as C
import os
import re

import pytest
import torch

from test_abi_host import BAD_PTR, BAD_PTR2, HEADER_DIR, INVALID, MISALIGNED, OK, UNSUPPORTED, \
    lib  # noqa: F401  (lib: the module fixture)

import rmsnorm_fwd_02_gb300 as R
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import dropout as D


def test_header_entry_points_are_exported_and_bound(lib):
    text = open(os.path.join(HEADER_DIR, "dropout_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^int (\w+)\s*\(", text, re.M)
    assert sorted(names) == ["dropout_train_bwd", "dropout_train_fwd",
                             "rmsnorm_dropout_train_bwd", "rmsnorm_dropout_train_fwd"]
    for name in names:
        assert hasattr(lib, name) and name in N.SIGNATURES


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID),
    (dict(y=None), INVALID),
    (dict(x=MISALIGNED), INVALID),
    (dict(y=MISALIGNED), INVALID),
    (dict(res=MISALIGNED), INVALID),
    (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID),
    (dict(n=-1), INVALID),
    (dict(n=1 << 40), UNSUPPORTED),
    (dict(p=-1e-9), INVALID),
    (dict(p=1.0000001), INVALID),
    (dict(p=float("nan")), INVALID),
    (dict(step=0x1004), INVALID),
    (dict(n=0), OK),                        # empty: nothing to do, no CUDA call
    (dict(n=0, x=None, y=None), OK),
    (dict(n=0, p=2.0), INVALID),
])
def test_dropout_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(x=BAD_PTR, res=None, y=BAD_PTR2, dtype=0, n=64, p=0.5, step=None) | kw
    assert lib.dropout_train_fwd(a["x"], a["res"], a["y"], a["dtype"], a["n"], a["p"], 1, 2,
                                 a["step"], None) == want
    if "res" not in kw:
        assert lib.dropout_train_bwd(a["x"], a["y"], a["dtype"], a["n"], a["p"], 1, 2, a["step"],
                                     None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(H=60), INVALID),
    (dict(H=0), INVALID),
    (dict(H=8200), UNSUPPORTED),
    (dict(T=-1), INVALID),
    (dict(nh=0), INVALID),
    (dict(T=1 << 31), UNSUPPORTED),
    (dict(wd=2), INVALID),
    (dict(x=None), INVALID),
    (dict(res=None), INVALID),
    (dict(w=None), INVALID),
    (dict(y=None), INVALID),
    (dict(h=None), INVALID),
    (dict(rstd=None), INVALID),
    (dict(res=MISALIGNED), INVALID),
    (dict(h=MISALIGNED), INVALID),
    (dict(rstd=BAD_PTR2 + 2), INVALID),
    (dict(s_tok=60), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(p=1.5), INVALID),
    (dict(p=float("nan")), INVALID),
    (dict(step=0x1001), INVALID),
    (dict(T=0), OK),
    (dict(T=0, x=None, res=None, y=None, h=None, rstd=None), OK),
    (dict(T=0, p=0.0), OK),
    (dict(T=0, w=None), INVALID),
])
def test_rmsnorm_dropout_fwd_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(x=BAD_PTR, res=BAD_PTR, w=BAD_PTR, wd=0, y=BAD_PTR2, h=BAD_PTR2, rstd=BAD_PTR2, T=4,
             nh=1, H=64, s_tok=64, eps=1e-6, p=0.5, step=None) | kw
    assert lib.rmsnorm_dropout_train_fwd(
        a["x"], a["res"], a["w"], a["wd"], a["y"], a["h"], a["rstd"], a["T"], a["nh"], a["H"],
        a["s_tok"], 64, a["eps"], a["p"], 1, 2, a["step"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(H=60), INVALID),
    (dict(H=8200), UNSUPPORTED),
    (dict(T=-1), INVALID),
    (dict(nh=0), INVALID),
    (dict(wd=2), INVALID),
    (dict(h=None), INVALID),
    (dict(dy=None), INVALID),
    (dict(rstd=None), INVALID),
    (dict(w=None), INVALID),
    (dict(dx=None), INVALID),
    (dict(dres=None), INVALID),
    (dict(dw=None), INVALID),
    (dict(dx=MISALIGNED), INVALID),
    (dict(dres=MISALIGNED), INVALID),
    (dict(dh=MISALIGNED), INVALID),
    (dict(rstd=BAD_PTR2 + 1), INVALID),
    (dict(ws=MISALIGNED), INVALID),
    (dict(det=2), INVALID),
    (dict(p=-0.1), INVALID),
    (dict(step=0x1002), INVALID),
])
def test_rmsnorm_dropout_bwd_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(h=BAD_PTR, dy=BAD_PTR, dh=None, rstd=BAD_PTR2, w=BAD_PTR, wd=0, dx=BAD_PTR2,
             dres=BAD_PTR2, dw=BAD_PTR2, ws=BAD_PTR, T=400, nh=1, H=64, p=0.5, step=None,
             det=1) | kw
    assert lib.rmsnorm_dropout_train_bwd(
        a["h"], a["dy"], a["dh"], a["rstd"], a["w"], a["wd"], a["dx"], a["dres"], a["dw"],
        a["ws"], 1 << 24, a["T"], a["nh"], a["H"], a["p"], 1, 2, a["step"], a["det"],
        None) == want


def test_torch_api_refuses_what_the_kernels_do_not_take():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: R.dropout_fwd(x, 0.5, 1), lambda: R.dropout_bwd(x, 0.5, 1),
                 lambda: R.rmsnorm_dropout_fwd(x, x, torch.ones(8), 0.5, 1),
                 lambda: R.rmsnorm_dropout_bwd(x, x, torch.ones(4), torch.ones(8), 0.5, 1)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.parametrize("args,error", [
    ((1.5, 1, 0, None), ValueError), ((-0.1, 1, 0, None), ValueError),
    ((float("nan"), 1, 0, None), ValueError), ((0.5, -1, 0, None), ValueError),
    ((0.5, 1 << 64, 0, None), ValueError), ((0.5, 1, 1 << 64, None), ValueError),
    ((0.5, 1.0, 0, None), ValueError), ((0.5, 1, 0, torch.zeros(1, dtype=torch.int64)), TypeError),
])
def test_generator_arguments_are_checked(args, error):
    with pytest.raises(error):
        D._generator(*args, torch.zeros(1))
