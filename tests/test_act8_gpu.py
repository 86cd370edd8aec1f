"""Activations held in 8 bits on the GPU against the FP64 oracle: packed bytes are equal, the norm
that keeps them and its backward within bounds from their roundings (tests/block_cases.py)."""
import numpy as np
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from block_cases import DEV, EPS, check, check_bwd, check_fwd, f64, normal
from oracle import act8 as OA
from rmsnorm_fwd_02_gb300 import _native as N

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
NARROW = DTYPES[:2]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,h", [(1, 1), (3, 7), (5, 8), (2, 31), (7, 32), (9, 33), (64, 256),
                                    (129, 264), (3, 2051), (33, 4096), (2, 16401)])
def test_packed_bytes(dtype, rows, h):
    x = normal(h, rows, h, dtype=dtype)
    x *= torch.exp2(torch.randint(-9, 9, (rows, 1), device=DEV)).to(dtype)
    p = R.act8_pack(x)
    assert p.shape == (rows, R.act8_row_bytes(h)) and p.dtype == torch.uint8
    assert np.array_equal(p.cpu().numpy(), OA.pack(f64(x)))
    held = OA.unpack(p.cpu().numpy(), h)
    for out in DTYPES:
        check(R.act8_unpack(p, h, out), held, 0 * held, "unpacked")
    if dtype != torch.float16:
        assert np.array_equal(f64(R.act8_unpack(p, h, torch.bfloat16)), held)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_packed_edges(dtype):
    info = torch.finfo(dtype)
    tiny = info.smallest_normal * info.eps
    rows = [[0.0], [-0.0], [tiny], [-tiny, info.smallest_normal], [info.max], [-info.max, 1.0],
            [127.5 / 64], [127 / 64, 63.5 / 64], [1.5, 0.5 / 64, 1.5 / 64, 2.5 / 64, -0.5 / 64],
            [float("inf"), 1.0], [float("nan")], [1.0, float("-inf"), float("nan")],
            [2.0 ** -14, 2.0 ** -24], [1e-39, 1e-40], [2.0 ** -120, 2.0 ** -127]]
    x = torch.zeros(len(rows), 40, dtype=dtype, device=DEV)
    for i, r in enumerate(rows):
        x[i, 3:3 + len(r)] = torch.tensor(r, dtype=torch.float64, device=DEV).to(dtype)
        x[i, 35] = 1.0                                   # the next block is its own
    p = R.act8_pack(x)
    assert np.array_equal(p.cpu().numpy(), OA.pack(f64(x)))
    held, got = OA.unpack(p.cpu().numpy(), 40), f64(R.act8_unpack(p, 40, dtype))
    # FP16's largest value is held as 2^16, which unpacks to FP16's largest
    want = np.where(np.abs(held) > info.max, np.copysign(info.max, held), held)
    keep = np.abs(want) >= tiny
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[keep], want[keep]) and (np.abs(got[~keep & ~np.isnan(want)]) <= tiny).all()
    assert (got[:, 35] == 1.0).all()
    wide = f64(R.act8_unpack(p, 40, torch.float32))
    assert np.array_equal(np.nan_to_num(wide, nan=7), np.nan_to_num(held, nan=7))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_strides_and_addresses(dtype):
    base = normal(3, 9, 5, 100, dtype=dtype)
    for x in (base[:, :, :64], base[:, 2, 8:72], base[:, :, 1:34], base[1:, 0], base[:1, :1, 3:4],
              base[0, 0, 5:], base[:, :, 96:]):
        want = R.act8_pack(x.contiguous())
        assert torch.equal(R.act8_pack(x), want)
        back = R.act8_unpack(want, x.shape[-1], dtype)
        assert back.shape == x.shape and torch.equal(R.act8_pack(back), want)   # held values stay
    p = R.act8_pack(base)
    at = torch.cat([p.new_zeros(5), p.flatten()])[5:].view_as(p)
    assert at.data_ptr() % 16 and torch.equal(R.act8_unpack(at, 100, dtype), R.act8_unpack(p, 100, dtype))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("h", list(range(1, 41)) + [47, 64, 190, 191])
def test_narrow_rows_at_every_alignment(dtype, h):
    flat = normal(h, 600 * h + 8, dtype=dtype)
    for off in (0, 1, 2, 3, 5):
        x = flat[off:off + 600 * h].view(600, h)
        p = R.act8_pack(x)
        want = OA.pack(f64(x))
        assert np.array_equal(p.cpu().numpy(), want)
        check(R.act8_unpack(p, h, dtype), OA.unpack(want, h), np.zeros((600, h)))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("h", [769, 772, 1024, 1027, 1032, 2055, 5001])
def test_wide_rows_at_every_alignment(dtype, h):
    # rows that start anywhere between two 16-byte vectors; rows, chunks and blocks end anywhere
    flat = normal(h, 9 * h + 8, dtype=dtype)
    for off in range(8):
        x = flat[off:off + 9 * h].view(9, h)
        p = R.act8_pack(x)
        want = OA.pack(f64(x))
        assert np.array_equal(p.cpu().numpy(), want)
        got = R.act8_unpack(p, h, dtype)
        check(got, OA.unpack(want, h), np.zeros((9, h)))
    # a narrower part of each row: what lies beside it is neither read into it nor written
    x = flat[:9 * h].view(9, h)[:, 3:h - 2]
    assert np.array_equal(R.act8_pack(x).cpu().numpy(), OA.pack(f64(x)))


def test_unpacked_rows_end_where_they_end():
    # through the C ABI into a guarded buffer: nothing before, behind or between is written
    for rows, h in ((3, 7), (300, 13), (257, 16), (700, 27), (256, 32), (5, 770), (4, 1031), (1, 4099)):
        p = R.act8_pack(normal(h, rows, h))
        for off in (0, 1, 5):
            buf = torch.full((rows * h + 24,), 7.0, dtype=torch.bfloat16, device=DEV)
            out = buf[8 + off:8 + off + rows * h]
            N.act8_train_unpack(p, out, N.ACT8_BF16, rows, h)
            assert torch.equal(out.view(rows, h), R.act8_unpack(p, h))
            assert (buf[:8 + off] == 7).all() and (buf[8 + off + rows * h:] == 7).all()


def test_empty_and_refusals():
    x = torch.empty(0, 40, device=DEV)
    p = R.act8_pack(x)
    assert p.shape == (0, R.act8_row_bytes(40)) and R.act8_unpack(p, 40).shape == (0, 40)
    with pytest.raises(ValueError, match="contiguous"):
        R.act8_pack(normal(1, 8, 8).t())
    with pytest.raises(ValueError, match="merge"):
        R.act8_pack(normal(1, 4, 6, 8).transpose(0, 1))
    with pytest.raises(ValueError, match="overlap"):
        R.act8_pack(normal(1, 8).expand(4, 8))
    with pytest.raises(ValueError, match="packed"):
        R.act8_unpack(p, 72)
    with pytest.raises(TypeError):
        R.act8_pack(torch.zeros(4, 8, dtype=torch.int32, device=DEV))


def test_rows_past_32_bits():
    rows, h = (1 << 20) + 3, 4104
    x = torch.zeros(rows, h, dtype=torch.bfloat16, device=DEV)   # 2^32 elements and more
    x[-2:] = normal(2, 2, h)
    x[1 << 19] = normal(3, h)
    p = R.act8_pack(x)
    for r in (1 << 19, rows - 2, rows - 1, 5):
        assert np.array_equal(p[r:r + 1].cpu().numpy(), OA.pack(f64(x[r:r + 1])))
    y = R.act8_unpack(p, h)
    assert torch.equal(y[-2:], R.act8_unpack(p[-2:], h)) and not y[7].any()


# ---- the norm that keeps its input in 8 bits -----------------------------------------------

SHAPES = [(1, 8), (3, 16), (700, 40), (257, 64), (65, 256), (700, 264), (33, 512), (300, 776),
          (260, 1536), (130, 2048), (300, 4096), (65, 5120), (310, 6144), (2, 7688), (270, 8192),
          (2501, 1536), (5003, 768), (1300, 2304)]


def case(rows, h, dtype, w_dtype, seed=0):
    x, res, dy, dh = (normal(seed + 10 * rows + h + i, rows, h, dtype=dtype) for i in range(4))
    return x, res, dy, dh, (1 + 0.1 * normal(seed + 5, h, dtype=torch.float32)).to(w_dtype)


@pytest.mark.parametrize("rows,h", SHAPES)
@pytest.mark.parametrize("dtype,w_dtype", [(torch.bfloat16, torch.bfloat16),
                                           (torch.bfloat16, torch.float32),
                                           (torch.float16, torch.float16)], ids=str)
def test_rmsnorm_act8(rows, h, dtype, w_dtype):
    x, res, dy, dh, w = case(rows, h, dtype, w_dtype)
    y, rstd, x8 = R.rmsnorm_act8_fwd(x, w)
    check_fwd((y, x, rstd, None), torch.zeros_like(x), x, w, None, None, 1.0, 1.0)
    assert torch.equal(x8, R.act8_pack(x))
    y, rstd, h8, out = R.rmsnorm_act8_fwd(x, w, residual=res)
    assert torch.equal(out, (x.float() + res.float()).to(dtype))
    assert torch.equal(h8, R.act8_pack(out))
    check_fwd((y, out, rstd, None), torch.zeros_like(x), out, w, None, None, 1.0, 1.0)
    for d in (None, dh):
        dx, dw = R.rmsnorm_act8_bwd(dy, h8, rstd, w, dh=d)
        check_bwd((dx, dx, dw, None, None), dy, d, None, h8, rstd, None, w, None, None, 1.0, 1.0)
    again = R.rmsnorm_act8_bwd(dy, h8, rstd, w, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rmsnorm_act8_is_rmsnorm_at_the_held_values():
    x, res, dy, dh, w = case(500, 1536, torch.bfloat16, torch.float32)
    y, rstd, h8, h = R.rmsnorm_act8_fwd(x, w, residual=res)
    y0, rstd0, h0 = R.rmsnorm_fwd(x, w, residual=res)
    assert torch.equal(h, h0)
    check(rstd, f64(rstd0), 40 * 2.0 ** -24 * f64(rstd0))
    assert (y.float() - y0.float()).abs().max() <= 2 * 2.0 ** -8 * y0.float().abs().max()
    # BF16 holds the values exactly, so rmsnorm_bwd can be asked at them
    dx, dw = R.rmsnorm_act8_bwd(dy, h8, rstd, w, dh=dh)
    dx0, dw0 = R.rmsnorm_bwd(dy, R.act8_unpack(h8, 1536), rstd, w, dh=dh)
    assert (dx.float() - dx0.float()).abs().max() <= 2 * 2.0 ** -8 * dx0.float().abs().max()
    assert ((dw - dw0).abs() <= 1e-4 + 1e-4 * dw0.abs()).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_bad_row_stays_alone(bad):
    x, res, dy, dh, w = case(40, 264, torch.bfloat16, torch.float32)
    good = R.rmsnorm_act8_fwd(x, w)
    x2 = x.clone()
    x2[17, 100] = bad
    y, rstd, x8 = R.rmsnorm_act8_fwd(x2, w)
    rows = torch.arange(40, device=DEV) != 17
    for p, q in zip((y, rstd, x8), good):
        assert torch.equal(p[rows], q[rows])
    assert y[17].isnan().any() and R.act8_unpack(x8, 264)[17, 96:128].isnan().all()
    dx = R.rmsnorm_act8_bwd(dy, x8, rstd, w)[0]
    assert torch.equal(dx[rows], R.rmsnorm_act8_bwd(dy, good[2], good[1], w)[0][rows])
    assert dx[17].isnan().all()


def test_strided_rows():
    base = normal(4, 60, 800)
    x, res = base[:, 16:280], normal(5, 60, 2, 264)[:, 1]
    w = normal(6, 264, dtype=torch.float32)
    for p, q in zip(R.rmsnorm_act8_fwd(x, w, residual=res),
                    R.rmsnorm_act8_fwd(x.contiguous(), w, residual=res.contiguous())):
        assert torch.equal(p, q)
    dy, dh = normal(7, 60, 800)[:, 8:272], normal(8, 264, 60).t()
    _, rstd, x8 = R.rmsnorm_act8_fwd(x, w)
    for p, q in zip(R.rmsnorm_act8_bwd(dy, x8, rstd, w, dh=dh),
                    R.rmsnorm_act8_bwd(dy.contiguous(), x8, rstd, w, dh=dh.contiguous())):
        assert torch.equal(p, q)
    for bad in (base[:, 4:268], base[:, ::2], base[:, 16:276]):
        with pytest.raises(ValueError):
            R.rmsnorm_act8_fwd(bad, w)


def test_no_rows():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.ones(64, device=DEV)
    y, rstd, x8 = R.rmsnorm_act8_fwd(x, w)
    assert y.shape == (0, 64) and x8.shape == (0, 80)
    dx, dw = R.rmsnorm_act8_bwd(y, x8, rstd, w)
    assert dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("dtype", NARROW, ids=str)
def test_autograd(dtype):
    x, res, dy, dh, w = case(77, 264, dtype, torch.float32)
    for t in (x, res, w):
        t.requires_grad_()
    y, h = R.rmsnorm_act8_train(x, w, residual=res)
    torch.autograd.backward([y, h], [dy, dh])
    _, rstd, h8, _ = R.rmsnorm_act8_fwd(x.detach(), w.detach(), residual=res.detach())
    dx, dw = R.rmsnorm_act8_bwd(dy, h8, rstd, w.detach(), dh=dh)
    assert torch.equal(x.grad, dx) and torch.equal(res.grad, dx) and torch.equal(w.grad, dw)
    x.grad = w.grad = None
    R.rmsnorm_act8_train(x, w).backward(dy)
    _, rstd, x8 = R.rmsnorm_act8_fwd(x.detach(), w.detach())
    dx, dw = R.rmsnorm_act8_bwd(dy, x8, rstd, w.detach())
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    x.grad = res.grad = w.grad = None
    R.rmsnorm_act8_train(x, w, residual=res)[1].backward(dh)   # h alone
    assert torch.equal(x.grad, dh) and not w.grad.any()


def test_no_wait_gave_up():
    assert N.rmsnorm_block_train_device_error() == 0
