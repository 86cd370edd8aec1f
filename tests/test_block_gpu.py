"""A block's boundary on the GPU against the FP64 oracle, element by element, within bounds from
the roundings (tests/block_cases.py)."""
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from block_cases import DEV, check_bwd, check_fwd, normal
from rmsnorm_fwd_02_gb300 import _native as N

pytestmark = pytest.mark.gpu

FORMS = [(True, True), (True, False), (False, True)]      # norm before, norm behind
SHAPES = [(1, 8, 1), (6, 16, 3), (720, 40, 5), (255, 64, 255), (64, 256, 2), (700, 264, 7), (60, 264, 10),
          (33, 512, 1), (310, 776, 31), (260, 1536, 2), (4 * 153, 2048, 153), (300, 4096, 5),
          (66, 5120, 3), (308, 6144, 4), (2, 7688, 2), (270, 8192, 6)]


def case(rows, h, n, pre, post, gate, dtype, w_dtype, seed=0):
    seed += 10 * rows + h
    c = dict(x=normal(seed, rows, h, dtype=dtype, scale=2.0),
             residual=normal(seed + 1, rows, h, dtype=dtype))
    one = lambda k: (1 + 0.1 * normal(seed + k, h, dtype=torch.float32)).to(w_dtype)  # noqa: E731
    f = dict(w_pre=one(2) if pre else None, w_post=one(3) if post else None, gate=None,
             scale=0.7, residual_scale=0.9)
    if gate == "row":
        f["gate"] = normal(seed + 4, h, dtype=w_dtype)
    elif gate == "sample":
        f["gate"] = normal(seed + 4, n, h, dtype=w_dtype)
    return c, f, normal(seed + 5, rows, h, dtype=dtype), normal(seed + 6, rows, h, dtype=dtype)


def run_case(c, f, dy, dh):
    out = R.rmsnorm_block_fwd(**c, **f)
    check_fwd(out, c["x"], c["residual"], f["w_pre"], f["w_post"], f["gate"], f["scale"],
              f["residual_scale"])
    y, h, rstd_pre, rstd_post, x8, h8 = R.rmsnorm_block_fwd(**c, **f, act8=True)
    for p, q in zip(out, (y, h, rstd_pre, rstd_post)):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))
    reads_x = f["w_post"] is not None or f["gate"] is not None
    assert (x8 is not None) == reads_x and (h8 is not None) == (f["w_pre"] is not None)
    if reads_x:
        assert torch.equal(x8, R.act8_pack(c["x"]))
    if f["w_pre"] is not None:
        assert torch.equal(h8, R.act8_pack(h))
    else:
        dy = None
    for x, kept in ((c["x"] if reads_x else None, h), (x8, h8)):
        for d in ((None, dh) if dy is not None else (dh,)):
            got = R.rmsnorm_block_bwd(dy, x, kept, rstd_pre, rstd_post, **f, dh=d)
            check_bwd(got, dy, d, x, kept if dy is not None else None, rstd_pre, rstd_post,
                      f["w_pre"], f["w_post"], f["gate"], f["scale"], f["residual_scale"])


@pytest.mark.parametrize("rows,h,n", SHAPES)
@pytest.mark.parametrize("pre,post", FORMS)
def test_block(rows, h, n, pre, post):
    for i, gate in enumerate(("none", "row", "sample")):
        dtype = (torch.bfloat16, torch.float16)[(h // 8 + i) % 2]
        w_dtype = (torch.float32, dtype)[(rows + i) % 2]
        run_case(*case(rows, h, n, pre, post, gate, dtype, w_dtype))


def test_many_rows():
    run_case(*case(40000, 64, 8, True, True, "row", torch.bfloat16, torch.float32))
    run_case(*case(40000, 264, 40000, True, True, "sample", torch.bfloat16, torch.float32))
    run_case(*case(20000, 520, 16, False, True, "sample", torch.float16, torch.float16))


def test_dtypes_mix_and_results_repeat():
    c, f, dy, dh = case(300, 264, 3, True, True, "sample", torch.bfloat16, torch.float32)
    f["gate"] = f["gate"].half()
    run_case(c, f, dy, dh)
    out = R.rmsnorm_block_fwd(**c, **f)
    first = R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)
    for _ in range(3):
        for p, q in zip(first, R.rmsnorm_block_bwd(dy, c["x"], *out[1:], **f, dh=dh)):
            assert torch.equal(p, q)


def test_no_wait_gave_up():
    assert N.rmsnorm_block_train_device_error() == 0
