"""The group norm entry points of the C-ABI library without a GPU: exported and bound; bad
arguments rejected before the first CUDA runtime call, in the C ABI and in the torch API; plans
that fit the kernels over a sweep of shapes; workspace sizes that depend on the shape only."""
import math
import os
import random
import re

import pytest
import torch

from test_abi_host import BAD_PTR, BAD_PTR2, HEADER_DIR, INVALID, MISALIGNED, OK, UNSUPPORTED, \
    lib  # noqa: F401  (lib: the module fixture)

import rmsnorm_fwd_02_gb300 as R
from rmsnorm_fwd_02_gb300 import _native as N
from rmsnorm_fwd_02_gb300 import groupnorm as GN

WORKSPACE = 3


def test_header_entry_points_are_exported_and_bound(lib):
    text = open(os.path.join(HEADER_DIR, "groupnorm_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^(?:int|size_t) (\w+)\s*\(", text, re.M)
    assert sorted(names) == ["groupnorm_train_bwd", "groupnorm_train_bwd_workspace_bytes",
                             "groupnorm_train_fwd", "groupnorm_train_fwd_workspace_bytes",
                             "groupnorm_train_launch_plan"]
    for name in names:
        assert hasattr(lib, name) and name in N.SIGNATURES


SIZES = [
    (dict(C=60), INVALID),
    (dict(C=0), INVALID),
    (dict(G=0), INVALID),
    (dict(G=3), INVALID),
    (dict(C=4104, G=8), UNSUPPORTED),
    (dict(dtype=1, C=4096, G=1), UNSUPPORTED),   # a group wider than 512 vectors
    (dict(N=-1), INVALID),
    (dict(S=-1), INVALID),
    (dict(S=0), INVALID),
    (dict(S=1 << 31), UNSUPPORTED),
    (dict(N=1 << 31, S=1), UNSUPPORTED),
    (dict(N=1 << 20, S=1 << 20), UNSUPPORTED),
    (dict(dtype=3), INVALID),
    (dict(wb=3), INVALID),
    (dict(act=3), INVALID),
    (dict(act=-1), INVALID),
    (dict(s_n=-8), INVALID),
    (dict(s_s=60), INVALID),
    (dict(dtype=1, s_s=66), INVALID),
]


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(x=None), INVALID),
    (dict(w=None), INVALID),
    (dict(b=None), INVALID),
    (dict(y=None), INVALID),
    (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID),
    (dict(x=MISALIGNED), INVALID),
    (dict(y=MISALIGNED), INVALID),
    (dict(w=BAD_PTR + 1), INVALID),
    (dict(wb=1, b=BAD_PTR + 2), INVALID),
    (dict(mean=BAD_PTR2 + 2), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(N=0), OK),
    (dict(N=0, S=0, x=None, y=None, mean=None, rstd=None), OK),
    (dict(N=0, w=None), INVALID),
    (dict(S=200000), WORKSPACE),                 # streamed: a workspace is due
    (dict(S=200000, ws=BAD_PTR, wsb=16), WORKSPACE),
    (dict(S=200000, ws=MISALIGNED, wsb=1 << 20), INVALID),
])
def test_fwd_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(x=BAD_PTR, dtype=0, w=BAD_PTR, b=BAD_PTR, wb=0, y=BAD_PTR2, mean=BAD_PTR2,
             rstd=BAD_PTR2, ws=None, wsb=0, N=2, S=9, C=64, G=8, s_n=640, s_s=64, eps=1e-5,
             act=1) | kw
    assert lib.groupnorm_train_fwd(
        a["x"], a["dtype"], a["w"], a["b"], a["wb"], a["y"], a["mean"], a["rstd"], a["ws"],
        a["wsb"], a["N"], a["S"], a["C"], a["G"], a["s_n"], a["s_s"], a["eps"], a["act"],
        None) == want


@pytest.mark.parametrize("kw,want", SIZES + [
    (dict(x=None), INVALID),
    (dict(dy=None), INVALID),
    (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID),
    (dict(w=None), INVALID),
    (dict(b=None), INVALID),
    (dict(dx=None), INVALID),
    (dict(dw=None), INVALID),
    (dict(db=None), INVALID),
    (dict(dy=MISALIGNED), INVALID),
    (dict(dx=MISALIGNED), INVALID),
    (dict(db=BAD_PTR2 + 1), INVALID),
    (dict(ws=None), WORKSPACE),
    (dict(wsb=64), WORKSPACE),
    (dict(ws=MISALIGNED), INVALID),
])
def test_bwd_rejects_before_any_cuda_call(lib, kw, want):
    a = dict(x=BAD_PTR, dy=BAD_PTR, dtype=0, mean=BAD_PTR2, rstd=BAD_PTR2, w=BAD_PTR, b=BAD_PTR,
             wb=0, dx=BAD_PTR2, dw=BAD_PTR2, db=BAD_PTR2, ws=BAD_PTR, wsb=1 << 30, N=2, S=9, C=64,
             G=8, s_n=640, s_s=64, act=1) | kw
    assert lib.groupnorm_train_bwd(
        a["x"], a["dy"], a["dtype"], a["mean"], a["rstd"], a["w"], a["b"], a["wb"], a["dx"],
        a["dw"], a["db"], a["ws"], a["wsb"], a["N"], a["S"], a["C"], a["G"], a["s_n"], a["s_s"],
        a["act"], None) == want


def test_plans_fit_the_kernels():
    rng = random.Random(3)
    seen = set()
    for _ in range(6000):
        dtype = rng.randrange(3)
        G = rng.choice([1, 2, 3, 4, 8, 16, 32, 64])
        c = G * int(2 ** rng.uniform(0, 12))
        C = c + (-c) % (8 * G // math.gcd(8, G))
        S = int(2 ** rng.uniform(0, 24))
        n = int(2 ** rng.uniform(0, 10))
        ev = 4 if dtype == 1 else 8
        least = C // G * (ev // math.gcd(C // G, ev)) // ev
        if C > 4096 or least > 512 or n * S * C >= 1 << 40:
            continue
        for bwd in (False, True):
            p = N.groupnorm_train_launch_plan(dtype, n, S, C, G, bwd)
            assert C % p["channels"] == 0 and p["channels"] % (C // G) == 0
            assert p["channels"] % ev == 0
            assert p["channels"] // ev <= p["threads"] <= 512 and p["threads"] % 32 == 0
            assert p["cluster_ctas"] in (1, 2, 4, 8) and p["smem"] <= 227 * 1024
            assert p["ctas"] % p["cluster_ctas"] == 0 and 0 < p["ctas"] < 1 << 31
            assert 1 <= p["chunks"] <= S and (p["on_chip"] == 0 or p["chunks"] == 1)
            assert p["units"] * p["chunks"] < 1 << 31 or p["on_chip"]
            assert p["on_chip"] or p["ctas"] <= 304
            assert 1 <= p["units"] <= n * (C // p["channels"])
            size = (N.groupnorm_train_bwd_workspace_bytes if bwd
                    else N.groupnorm_train_fwd_workspace_bytes)(dtype, n, S, C, G)
            if not bwd:
                assert (size == 0) == (p["on_chip"] == 1)
            # never more than the activation itself (and one wave's column sums)
            assert size <= max(n * S * C * (4 if dtype == 1 else 2), 2432 * 2 * C * 4)
            seen.add((bwd, p["on_chip"], p["cluster_ctas"]))
    assert {(d, 1, k) for d in (False, True) for k in (1, 2, 4, 8)} <= seen
    assert {(d, 0, 1) for d in (False, True)} <= seen


def test_torch_api_refuses_what_the_kernels_do_not_take():
    x = torch.zeros(2, 5, 16, dtype=torch.bfloat16)
    w = torch.ones(16)
    for call in (lambda: R.groupnorm_fwd(x, w, w, 4),
                 lambda: R.groupnorm_bwd(x, x, torch.zeros(2, 4), torch.ones(2, 4), w, w, 4)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="act"):
        GN._act("relu6")
