"""The builds of the block boundary's kernels that large batches take at real widths (several vectors
a thread, uneven last vectors) against the FP64 oracle, in both activation types, within the bounds
of block_cases.py; the column sums' with the additions of the launch that made them.

Additions of a column sum: a team's lane adds its rows one after another.  With one sample a CTA's
teams take its ring slots in turns: of a CTA's rows a team has at most ceil(slots / teams) slots of
p["rows"] rows, `side` of which lie side by side in a warp and have sums of their own.  With
several samples a team has a run of rows, which it takes in pieces that end with a sample.  The few
additions behind that (lanes, teams, CTAs) are in block_cases.py's 8."""
import pytest
import torch

import block_cases
import rmsnorm_fwd_02_gb300 as R
from block_builds import NO_GATE, NO_POST, NO_PRE, NORM8, ONE
from block_cases import DEV, U, check_bwd, check_fwd
from rmsnorm_fwd_02_gb300 import _native as N
from test_block_gpu import FORMS, case

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8), (1830, 96), (930, 384), (310, 1000), (620, 768), (160, 1792), (160, 2304),
          (160, 3584), (20, 7000)]           # each a batch of two or ten samples
MANY = [(720, 40), (612, 2048), (270, 8192)]  # shapes of test_block_gpu.py


def up(a, b):
    return -(-a // b)


def chain(p, rows, n):
    """Most additions one after another in a team's sum of a column."""
    if n > 1:
        return up(rows, p["ctas"] * p["teams"]) + 1
    side = 32 // p["row_threads"] if p["row_threads"] < 32 else 1
    slots = up(up(rows, p["ctas"]), p["rows"])
    return up(slots, p["teams"]) * (p["rows"] // side)


def sums_of(monkeypatch, form):
    """block_cases.check_bwd with the plan of the kernel that `form` names."""
    def rows_of(rows, h, n, packed):
        p = N.rmsnorm_block_train_launch_plan(rows, h, n, True, packed, form)
        return chain(p, rows, n)
    monkeypatch.setattr(block_cases, "team_rows", rows_of)


@pytest.mark.parametrize("rows,h", SHAPES)
@pytest.mark.parametrize("pre,post", FORMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_builds(monkeypatch, rows, h, pre, post, dtype):
    gates = ("none", "row", "sample")
    for gate in gates if rows > 1 else gates[:2]:
        w_dtype = torch.float32 if gate == "row" else dtype
        c, f, dy, dh = case(rows, h, 10 if rows % 10 == 0 else 1, pre, post, gate, dtype, w_dtype)
        y, out, r2, r1, x8, h8 = R.rmsnorm_block_fwd(**c, **f, act8=True)
        check_fwd((y, out, r2, r1), c["x"], c["residual"], f["w_pre"], f["w_post"], f["gate"],
                  f["scale"], f["residual_scale"])
        for p, q in zip((y, out, r2, r1), R.rmsnorm_block_fwd(**c, **f)):
            assert (p is None and q is None) or torch.equal(p, q)
        assert x8 is None or torch.equal(x8, R.act8_pack(c["x"]))
        assert h8 is None or torch.equal(h8, R.act8_pack(out))
        x = c["x"] if post or gate != "none" else None
        for kept in ((x, out), (x8, h8)):
            for d in (None, dh) if pre else (dh,):
                flags = (not post) * NO_POST | (not pre) * NO_PRE | (gate == "none") * NO_GATE | \
                    (d is None) * ONE
                sums_of(monkeypatch, flags)
                grads = R.rmsnorm_block_bwd(dy if pre else None, *kept, r2, r1, **f, dh=d)
                check_bwd(grads, dy if pre else None, d, kept[0], kept[1] if pre else None, r2, r1,
                          f["w_pre"], f["w_post"], f["gate"], f["scale"], f["residual_scale"])


@pytest.mark.parametrize("rows,h", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_norm8_builds(monkeypatch, rows, h, dtype):
    c, f, dy, dh = case(rows, h, 1, True, False, "none", dtype, torch.float32)
    x, res, w = c["x"], c["residual"], f["w_pre"]
    y, rstd, h8, out = R.rmsnorm_act8_fwd(x, w, residual=res)
    assert torch.equal(out, (x.float() + res.float()).to(dtype))
    assert torch.equal(h8, R.act8_pack(out))
    check_fwd((y, out, rstd, None), torch.zeros_like(x), out, w, None, None, 1.0, 1.0)
    for d in (None, dh):
        sums_of(monkeypatch, NORM8 | (d is None) * ONE)
        dx, dw = R.rmsnorm_act8_bwd(dy, h8, rstd, w, dh=d)
        check_bwd((dx, dx, dw, None, None), dy, d, None, h8, rstd, None, w, None, None, 1.0, 1.0)


@pytest.mark.parametrize("packed", [False, True])
def test_long_column_sums(packed):
    """dw of 400000 rows is as near as its additions allow: each errs by at most U of the partial
    sum that it forms, and the partial sums of values of both signs stay far below the sum of
    magnitudes that a bound for any values would take.  The partial sums are those of the plan."""
    rows, h, cols = 400000, 1024, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    normal = lambda: torch.randn(rows, h, device=DEV, generator=g).bfloat16()  # noqa: E731
    x, dy, w = normal(), normal(), torch.ones(h, device=DEV)
    if packed:
        _, rstd, kept = R.rmsnorm_act8_fwd(x, w)
        dw = R.rmsnorm_act8_bwd(dy, kept, rstd, w)[1]
        x = R.act8_unpack(kept, h)
        flags = NORM8 | ONE
    else:
        _, _, rstd, _ = R.rmsnorm_block_fwd(x, torch.zeros_like(x), w)
        dw = R.rmsnorm_block_bwd(dy, None, x, rstd, None, w)[2]
        flags = NO_POST | NO_GATE | ONE
    p = N.rmsnorm_block_train_launch_plan(rows, h, 1, True, packed, flags)
    assert p["row_threads"] >= 32
    terms = dy[:, :cols].double() * (x[:, :cols].double() * rstd.double()[:, None])
    err = 2 * U * terms.abs().sum(0)        # h * rstd is rounded, dy times it in the fma not
    longest = 0
    for cta in range(p["ctas"]):
        own = terms[cta * rows // p["ctas"]:(cta + 1) * rows // p["ctas"]]
        slot = torch.arange(len(own), device=DEV) // p["rows"]
        for team in range(p["teams"]):
            mine = own[slot % p["teams"] == team]
            longest = max(longest, len(mine))
            err += U * mine.cumsum(0).abs().sum(0)
    want = terms.sum(0)
    assert longest <= chain(p, rows, 1)
    err += U * (want.abs() + err)           # the joined sum's rounding
    far = ((dw[:cols].double() - want).abs() / err).max()
    assert far <= 1, far
    # a bound for any values would allow this much more
    assert (err < 0.2 * longest * U * terms.abs().sum(0)).all()


def test_no_wait_gave_up():
    assert N.rmsnorm_block_train_device_error() == 0
