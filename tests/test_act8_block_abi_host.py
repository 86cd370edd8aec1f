"""The entry points of 8-bit activations and of a block's boundary without a GPU: declared, exported
and bound; bad arguments rejected before the first CUDA runtime call, in the C ABI and in the
torch API; workspace sizes and launch plans over every width; the headers from plain C."""
import os
import re
import subprocess

import pytest
import torch

from test_abi_host import BAD_PTR, BAD_PTR2, HEADER_DIR, INVALID, MISALIGNED, OK, UNSUPPORTED, \
    lib  # noqa: F401  (lib: the module fixture)

import rmsnorm_fwd_02_gb300 as R
from oracle import act8 as OA
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import block as B

A, P = BAD_PTR, BAD_PTR2     # addresses of inputs and of outputs, never touched


@pytest.mark.parametrize("header,want", [
    ("act8_train.h", ["act8_train_pack", "act8_train_row_bytes", "act8_train_unpack",
                      "rmsnorm_act8_train_bwd", "rmsnorm_act8_train_bwd_workspace_bytes",
                      "rmsnorm_act8_train_fwd"]),
    ("block_train.h", ["rmsnorm_block_train_bwd", "rmsnorm_block_train_bwd_workspace_bytes",
                       "rmsnorm_block_train_device_error", "rmsnorm_block_train_fwd",
                       "rmsnorm_block_train_launch_plan"]),
])
def test_header_entry_points_are_exported_and_bound(lib, header, want):
    text = open(os.path.join(HEADER_DIR, header)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:int|size_t|int64_t) (\w+)\s*\(", text, re.M)
    assert sorted(names) == want
    for name in names:
        assert hasattr(lib, name) and name in N.SIGNATURES


@pytest.mark.parametrize("h", list(range(1, 100)) + [2051, 8192, 1 << 30])
def test_row_bytes(lib, h):
    assert N.act8_train_row_bytes(h) == R.act8_row_bytes(h) == OA.row_bytes(h)


def test_row_bytes_of_no_row(lib):
    assert [N.act8_train_row_bytes(h) for h in (0, -5, (1 << 30) + 1)] == [0, 0, 0]
    with pytest.raises(ValueError):
        R.act8_row_bytes(0)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(p=None), INVALID), (dict(p=MISALIGNED), INVALID),
    (dict(x=A + 1), INVALID), (dict(dtype=1, x=A + 2), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID), (dict(h=0), INVALID),
    (dict(h=(1 << 30) + 1), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(rows=0), OK), (dict(rows=0, x=None, p=None), OK),
])
def test_pack_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(x=A, p=P, dtype=0, rows=4, h=64) | kw
    assert lib.act8_train_pack(a["x"], a["dtype"], a["p"], a["rows"], a["h"], a["h"], None) == want
    assert lib.act8_train_unpack(a["p"], a["x"], a["dtype"], a["rows"], a["h"], None) == want


def test_pack_rejects_a_negative_stride(lib):
    assert lib.act8_train_pack(A, 0, P, 4, 64, -64, None) == INVALID


FWD8 = dict(x=A, res=None, dtype=0, w=A, wd=1, y=P, h=None, rstd=P, packed=P, R=4, H=64, sx=64,
            sr=64, eps=1e-6)


@pytest.mark.parametrize("kw,want", [
    (dict(H=60), INVALID), (dict(H=0), INVALID), (dict(H=8200), UNSUPPORTED), (dict(R=-1), INVALID),
    (dict(R=1 << 31), UNSUPPORTED), (dict(dtype=1), INVALID), (dict(dtype=3), INVALID),
    (dict(wd=3), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(rstd=None), INVALID), (dict(packed=None), INVALID), (dict(res=A), INVALID),
    (dict(h=P), INVALID), (dict(x=MISALIGNED), INVALID), (dict(packed=MISALIGNED), INVALID),
    (dict(rstd=P + 2), INVALID), (dict(sx=60), INVALID), (dict(sx=-64), INVALID),
    (dict(res=A, h=P, sr=4), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(R=0), OK), (dict(R=0, x=None, y=None, rstd=None, packed=None), OK),
    (dict(R=0, w=None), INVALID),
])
def test_rmsnorm_act8_fwd_rejects_before_any_cuda_call(lib, kw, want):
    a = FWD8 | kw
    assert lib.rmsnorm_act8_train_fwd(*a.values(), None) == want


BWD8 = dict(packed=A, dy=A, dh=None, dtype=0, rstd=A, w=A, wd=1, dx=P, dw=P, ws=P, wsb=1 << 24, R=400,
            H=64)


@pytest.mark.parametrize("kw,want", [
    (dict(H=60), INVALID), (dict(H=8200), UNSUPPORTED), (dict(R=-1), INVALID), (dict(dtype=1), INVALID),
    (dict(wd=-1), INVALID), (dict(packed=None), INVALID), (dict(dy=None), INVALID),
    (dict(rstd=None), INVALID), (dict(w=None), INVALID), (dict(dx=None), INVALID),
    (dict(dw=None), INVALID), (dict(packed=MISALIGNED), INVALID), (dict(dh=MISALIGNED), INVALID),
    (dict(ws=MISALIGNED), INVALID), (dict(rstd=A + 1), INVALID), (dict(dw=P + 2), INVALID),
])
def test_rmsnorm_act8_bwd_rejects_before_any_cuda_call(lib, kw, want):
    a = BWD8 | kw
    assert lib.rmsnorm_act8_train_bwd(*a.values(), None) == want


FWD = dict(x=A, res=A, dtype=0, w_pre=A, w_post=A, wd=1, gate=A, gd=1, N=2, y=P, h=P, r_pre=P,
           r_post=P, x8=None, h8=None, R=4, H=64, sx=64, sr=64, scale=1.0, rscale=1.0, eps=1e-6)
NO_PRE = dict(w_pre=None, y=None, r_pre=None)
NO_POST = dict(w_post=None, r_post=None)


@pytest.mark.parametrize("kw,want", [
    (dict(H=12), INVALID), (dict(H=8200), UNSUPPORTED), (dict(R=1 << 31), UNSUPPORTED),
    (dict(N=0), INVALID), (dict(N=3), INVALID), (dict(gate=None), INVALID), (dict(gd=4), INVALID),
    (dict(dtype=1), INVALID), (dict(wd=5), INVALID), (dict(x=None), INVALID), (dict(res=None), INVALID),
    (dict(h=None), INVALID), (dict(y=None), INVALID), (dict(r_pre=None), INVALID),
    (dict(r_post=None), INVALID), (dict(w_pre=None), INVALID), (dict(w_post=None), INVALID),
    (NO_PRE | NO_POST, INVALID), (dict(x8=P), INVALID), (dict(h8=P), INVALID),
    (NO_PRE | dict(h8=P), INVALID), (NO_POST | dict(gate=None, N=1, x8=P, h8=P), INVALID),
    (dict(gate=MISALIGNED), INVALID), (dict(w_post=MISALIGNED), INVALID),
    (dict(h=MISALIGNED), INVALID), (dict(r_post=P + 2), INVALID), (dict(sx=65), INVALID),
    (dict(sr=-8), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(rscale=float("nan")), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(R=0), OK), (dict(R=0, x=None, res=None, y=None, h=None, r_pre=None, r_post=None), OK),
])
def test_block_fwd_rejects_before_any_cuda_call(lib, kw, want):
    a = FWD | kw
    assert lib.rmsnorm_block_train_fwd(*a.values(), None) == want


BWD = dict(dy=A, dh=None, x=A, h=A, packed=0, dtype=0, r_pre=A, r_post=A, w_pre=A, w_post=A, wd=1,
           gate=A, gd=1, N=2, dx=P, dres=P, dw_pre=P, dw_post=P, dgate=P, ws=P, wsb=1 << 24, R=400,
           H=64, sx=64, scale=1.0, rscale=1.0)


@pytest.mark.parametrize("kw,want", [
    (dict(H=12), INVALID), (dict(H=8200), UNSUPPORTED), (dict(N=3), INVALID), (dict(N=-1), INVALID),
    (dict(packed=2), INVALID), (dict(dtype=1), INVALID), (dict(wd=3), INVALID), (dict(gd=3), INVALID),
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(h=None), INVALID),
    (dict(r_pre=None), INVALID), (dict(r_post=None), INVALID), (dict(dx=None), INVALID),
    (dict(dres=None), INVALID), (dict(dw_pre=None), INVALID), (dict(dw_post=None), INVALID),
    (dict(dgate=None), INVALID), (dict(w_pre=None), INVALID), (dict(w_post=None), INVALID),
    (dict(gate=None), INVALID), (dict(w_pre=None, dw_pre=None, dy=None), INVALID),  # dh is needed
    (dict(w_pre=None, dw_pre=None, w_post=None, dw_post=None, dy=None, dh=A), INVALID),
    (dict(dh=MISALIGNED), INVALID), (dict(x=MISALIGNED), INVALID), (dict(ws=MISALIGNED), INVALID),
    (dict(dgate=P + 2), INVALID), (dict(r_pre=A + 1), INVALID), (dict(sx=12), INVALID),
    (dict(scale=float("nan")), INVALID),
])
def test_block_bwd_rejects_before_any_cuda_call(lib, kw, want):
    a = BWD | kw
    assert lib.rmsnorm_block_train_bwd(*a.values(), None) == want


def test_plans_fit_the_device(lib):
    for h in list(range(8, 700, 8)) + list(range(704, 8193, 72)) + [8192]:
        for rows in (1, 7, 152, 153, 2000, 100000, (1 << 31) - (1 << 16)):
            for backward in (0, 1):
                for packed in (0, 1):
                    p = N.rmsnorm_block_train_launch_plan(rows, h, 1, backward, packed)
                    assert p["smem"] <= 227 * 1024 and 1 <= p["ctas"] <= 152
                    assert p["threads"] <= (256 if backward and not packed else 384)
                    assert p["stages"] >= 2
                    assert 8 * p["vectors"] * p["row_threads"] >= h
                    side = 32 // p["row_threads"] if p["row_threads"] < 32 else 1
                    assert p["threads"] == p["teams"] * side * p["row_threads"]
                    assert p["rows"] % side == 0


def test_workspace_sizes(lib):
    size = N.rmsnorm_block_train_bwd_workspace_bytes
    for h in (8, 256, 1536, 4096, 8192):
        for rows in (1, 100, 1000, 100000):
            p = N.rmsnorm_block_train_launch_plan(rows, h, 1, 1, 0)
            assert size(rows, h, 1) >= 8 * p["ctas"] * h
            assert size(rows, h, rows) >= 4 * h * (p["ctas"] + p["ctas"] * p["teams"] + rows - 1)
            assert 0 < N.rmsnorm_act8_train_bwd_workspace_bytes(rows, h) <= 4 * 152 * h
    assert size(0, 64, 1) == size(10, 60, 1) == size(10, 64, 3) == size(10, 64, 0) == 0
    assert N.rmsnorm_act8_train_bwd_workspace_bytes(0, 64) == 0


def test_torch_api_refuses_what_the_kernels_do_not_take():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    w, r = torch.ones(8), torch.ones(4)
    p = torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: R.act8_pack(x), lambda: R.act8_unpack(p, 8),
                 lambda: R.rmsnorm_act8_fwd(x, w), lambda: R.rmsnorm_act8_bwd(x, p, r, w),
                 lambda: R.rmsnorm_block_fwd(x, x, w), lambda: R.rmsnorm_block_bwd(x, x, x, r, r, w)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="dy"):
        R.rmsnorm_block_bwd(None, x, x, r, r, w)
    with pytest.raises(ValueError, match="dh"):
        R.rmsnorm_block_bwd(None, x, None, None, r, None, w)


W, G = torch.ones(8), torch.ones(2, 8)


@pytest.mark.parametrize("args,error", [
    ((4, 8, None, None, None, 1.0, 1.0), ValueError),
    ((4, 8, W, W.half(), None, 1.0, 1.0), TypeError),
    ((4, 8, W.double(), None, None, 1.0, 1.0), TypeError),
    ((4, 8, torch.ones(9), None, None, 1.0, 1.0), ValueError),
    ((4, 8, torch.ones(1, 8), None, None, 1.0, 1.0), ValueError),
    ((5, 8, W, None, G, 1.0, 1.0), ValueError),
    ((4, 8, W, None, torch.ones(0, 8), 1.0, 1.0), ValueError),
    ((4, 8, W, None, torch.ones(2, 1, 8), 1.0, 1.0), ValueError),
    ((4, 8, W, None, torch.ones(4), 1.0, 1.0), ValueError),
    ((4, 8, W, None, G.int(), 1.0, 1.0), TypeError),
    ((4, 8, W, None, None, float("inf"), 1.0), ValueError),
    ((4, 8, W, None, None, 1.0, float("nan")), ValueError),
])
def test_block_factors_are_checked(args, error):
    with pytest.raises(error):
        B._factors(*args)


PROGRAM = r"""
#include <stdio.h>
#include "act8_train.h"
#include "block_train.h"

int main(void) {
  int64_t p[BLOCK_PLAN_FIELDS];
  int i;
  if (rmsnorm_block_train_launch_plan(4096, 1536, 4, 1, 1, p, BLOCK_PLAN_FIELDS) != RMSN_OK) return 1;
  printf("plan");
  for (i = 0; i < BLOCK_PLAN_FIELDS; ++i) printf(" %lld", (long long)p[i]);
  printf("\n");
  printf("row %lld\n", (long long)act8_train_row_bytes(2051));
  printf("ws %zu\n", rmsnorm_block_train_bwd_workspace_bytes(4096, 1536, 4));
  printf("ws8 %zu\n", rmsnorm_act8_train_bwd_workspace_bytes(4096, 1536));
  printf("none %d\n", act8_train_pack(NULL, ACT8_FP32, NULL, 0, 7, 7, NULL));
  printf("null %d\n", act8_train_unpack(NULL, NULL, ACT8_FP16, 8, 7, NULL));
  printf("wide %d\n", rmsnorm_act8_train_fwd(NULL, NULL, ACT8_BF16, NULL, ACT8_FP32, NULL, NULL, NULL,
                                            NULL, 4, 8200, 8200, 8200, 1e-6f, NULL));
  printf("bnull %d\n", rmsnorm_block_train_bwd(NULL, NULL, NULL, NULL, 0, ACT8_BF16, NULL, NULL, NULL,
                                              NULL, ACT8_FP32, NULL, 0, 1, NULL, NULL, NULL, NULL,
                                              NULL, NULL, 0, 4, 64, 64, 1.f, 1.f, NULL));
  return 0;
}
"""


def test_c_program_links_and_sees_the_bindings_values(tmp_path):
    from rmsnorm_fwd_02_gb300 import build as BB
    libdir = os.path.dirname(BB.build())
    src, exe = tmp_path / "abi.c", tmp_path / "abi"
    src.write_text(PROGRAM)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", HEADER_DIR,
                    str(src), "-o", str(exe), "-L", libdir, "-lrmsnorm_train",
                    f"-Wl,-rpath,{libdir}"], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    got = dict(line.split(" ", 1) for line in out.strip().splitlines())
    plan = N.rmsnorm_block_train_launch_plan(4096, 1536, 4, 1, 1)
    assert [int(v) for v in got["plan"].split()] == [plan[k] for k in N.BLOCK_PLAN_FIELDS]
    assert int(got["row"]) == OA.row_bytes(2051)
    assert int(got["ws"]) == N.rmsnorm_block_train_bwd_workspace_bytes(4096, 1536, 4)
    assert int(got["ws8"]) == N.rmsnorm_act8_train_bwd_workspace_bytes(4096, 1536)
    assert [int(got[k]) for k in ("none", "null", "wide", "bnull")] == [OK, INVALID, UNSUPPORTED, INVALID]
