"""The dropout entry points on the GPU against the FP64 oracle (oracle/dropout.py), element by
element.

Tolerances, from the roundings alone (u = eps / 2 of the output type, 2^-24 FP32's):
  y = dropout(x) [+ residual] is one FP32 multiply or fma with scale rounded to FP32, then one
  rounding to the output type: with d = 2^-24 (|x scale| + |e| + |x scale| 2^-23) the FP32
  value is within d of the exact e, and y within d + u (|e| + d) (+ half the type's smallest
  subnormal).  Dropped elements of a plain dropout are exactly 0.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from oracle import dropout as OD
from rmsnorm_fwd_02_gb300 import _native as N

pytestmark = pytest.mark.gpu

DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
U32 = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def check_sum(y, x, p, seed, counter, residual=None):
    """y against the oracle's [residual +] dropout(x), within the module's tolerance."""
    x64 = f64(x)
    e = OD.fwd(x64, p, seed, counter, None if residual is None else f64(residual))
    xs = np.abs(OD.fwd(x64, p, seed, counter))
    d = U32 * (xs + np.abs(e) + xs * 2.0 ** -23)
    info = torch.finfo(y.dtype)
    u = 0.0 if y.dtype == torch.float32 else info.eps / 2
    tiny = info.smallest_normal * info.eps / 2
    err = np.abs(f64(y) - e)
    assert (err <= d + u * (np.abs(e) + d) + tiny).all(), err.max()
    return e


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2043, 8192, 8193, 100003])
@pytest.mark.parametrize("with_residual", [False, True])
def test_dropout_values(dtype, n, with_residual):
    for p in (0.0, 0.1, 0.5, 0.9, 1.0):
        seed, offset = 0x0123456789ABCDEF + n, (1 << 40) + 3
        x = normal(n, n, dtype=dtype)
        r = normal(n + 1, n, dtype=dtype) if with_residual else None
        y = R.dropout_fwd(x, p, seed, offset, residual=r)
        check_sum(y, x, p, seed, offset, r)
        k = OD.keep(n, p, seed, offset)
        got = f64(y)
        if with_residual:
            assert np.array_equal(got[~k], f64(r)[~k])
        else:
            assert not got[~k].any()
            assert torch.equal(R.dropout_bwd(x, p, seed, offset), y)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_dropped_infinities_and_nan_do_not_pass(dtype):
    n, p, seed = 4099, 0.5, 77
    k = OD.keep(n, p, seed, 0)
    x = torch.full((n,), float("nan"), dtype=dtype, device=DEV)
    x[1::3] = float("inf")
    r = normal(3, n, dtype=dtype)
    y = R.dropout_fwd(x, p, seed)
    assert not f64(y)[~k].any() and not np.isfinite(f64(y)[k]).any()
    y = R.dropout_fwd(x, p, seed, residual=r)
    assert np.array_equal(f64(y)[~k], f64(r)[~k]) and not np.isfinite(f64(y)[k]).any()
    assert not f64(R.dropout_bwd(x, 1.0, seed)).any()


@pytest.mark.parametrize("seed,offset,step", [
    (0, 0, None), ((1 << 64) - 1, (1 << 64) - 1, None), (1 << 32, 1 << 32, 5),
    (5, (1 << 64) - 2, 9), (5, 3, -1),
])
def test_seed_offset_and_step_words(seed, offset, step):
    n, p = 1003, 0.3
    x = torch.ones(n, dtype=torch.float32, device=DEV)
    s = None if step is None else torch.tensor([step], dtype=torch.int64, device=DEV)
    y = R.dropout_fwd(x, p, seed, offset, step=s)
    assert np.array_equal(f64(y) != 0, OD.keep(n, p, seed, (offset + (step or 0)) % (1 << 64)))


def test_elements_past_32_bits():
    n = (1 << 32) + 8 * 1000 + 5
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    y = R.dropout_fwd(x, 0.5, 11, 13)
    for first in (0, (1 << 32) - 4096, n - 5 - 4096):
        part = y[first:first + 4101 if first + 4101 <= n else n]
        assert np.array_equal(f64(part) != 0, OD.keep(part.numel(), 0.5, 11, 13, first))


def test_shapes_and_empty_tensors():
    x = normal(1, 3, 5, 7, dtype=torch.float16)
    y = R.dropout_fwd(x, 0.25, 9)
    assert y.shape == x.shape and torch.equal(y.view(-1), R.dropout_fwd(x.view(-1), 0.25, 9))
    e = torch.empty(0, 4, device=DEV)
    assert R.dropout_fwd(e, 0.5, 1).shape == (0, 4) and R.dropout_bwd(e, 0.5, 1).shape == (0, 4)
    with pytest.raises(ValueError, match="contiguous"):
        R.dropout_fwd(normal(2, 8, 8).t(), 0.5, 1)
    with pytest.raises(ValueError, match="residual"):
        R.dropout_fwd(x, 0.5, 1, residual=x.float())
    with pytest.raises(N.RmsnError):             # 2-byte aligned
        R.dropout_fwd(normal(2, 17)[1:], 0.5, 1)
    t = normal(2, 8, 16)
    assert torch.equal(R.dropout_bwd(t.t(), 0.5, 1), R.dropout_bwd(t.t().contiguous(), 0.5, 1))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_tensors_at_any_address(dtype):
    # a gradient that is a slice of another tensor starts anywhere: the same values
    at = lambda t: torch.cat([t.new_zeros(1), t])[1:]  # noqa: E731
    x, res = (normal(i, 1003, dtype=dtype) for i in (1, 2))
    assert at(x).is_contiguous() and at(x).data_ptr() % 16
    assert torch.equal(R.dropout_fwd(x, 0.3, 4, residual=at(res)),
                       R.dropout_fwd(x, 0.3, 4, residual=res))
    assert torch.equal(R.dropout_bwd(at(x), 0.3, 4), R.dropout_bwd(x, 0.3, 4))
    x.requires_grad_()
    y = torch.cat([res[:5], R.dropout_train(x, 0.3, 4)])
    g = normal(3, 1008, dtype=dtype)
    y.backward(g)
    assert torch.equal(x.grad, R.dropout_bwd(g[5:].clone(), 0.3, 4))


def test_rmsnorm_dropout_gradients_at_any_address():
    at = lambda t: torch.cat([t.new_zeros(5), t.flatten()])[5:].view_as(t)  # noqa: E731
    x, res, dy, dh, w = rms_case(300, 264, 8, torch.float32)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, 0.2, 6)
    for p, q in zip(R.rmsnorm_dropout_bwd(at(dy), h, rstd, w, 0.2, 6, dh=at(dh)),
                    R.rmsnorm_dropout_bwd(dy, h, rstd, w, 0.2, 6, dh=dh)):
        assert torch.equal(p, q)


def test_residual_that_is_x():
    x = normal(5, 777)
    x.requires_grad_()
    y = R.dropout_train(x, 0.4, 9, residual=x)
    y.backward(torch.ones_like(y))
    assert torch.equal(y.detach(), R.dropout_fwd(x.detach(), 0.4, 9, residual=x.detach().clone()))
    one = R.dropout_bwd(torch.ones_like(y), 0.4, 9)
    assert torch.equal(x.grad, one + 1)


def test_dropout_autograd():
    x = normal(4, 33, 65).requires_grad_()
    r = normal(5, 33, 65).requires_grad_()
    dy = normal(6, 33, 65)
    step = torch.tensor([4], dtype=torch.int64, device=DEV)
    y = R.dropout_train(x, 0.3, 21, 2, step, r)
    assert torch.equal(y, R.dropout_fwd(x.detach(), 0.3, 21, 6, residual=r.detach()))
    y.backward(dy)
    assert torch.equal(x.grad, R.dropout_bwd(dy, 0.3, 21, 6)) and torch.equal(r.grad, dy)
    y = R.dropout_train(x, 0.3, 21, 2, step)
    step.add_(1)                                  # the backward would draw another mask
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy)


# ---- the residual norm with dropout -------------------------------------------------------

# every forward and backward shape class, sub-warp and whole-warp groups, ragged widths; few
# rows (the one-launch backward) and more than 256
SHAPES = [(1, 8), (3, 16), (300, 8), (257, 64), (65, 256), (700, 264), (33, 512), (300, 768),
          (260, 1000), (300, 1536), (130, 2048), (300, 4096), (65, 5120), (300, 6144), (2, 7688),
          (270, 8192)]


def rms_case(T, H, seed, w_dtype):
    x, res, dy, dh = (normal(seed + i, T, H) for i in range(4))
    w = (1 + 0.1 * normal(seed + 9, H, dtype=torch.float32)).to(w_dtype)
    return x, res, dy, dh, w


def half_ulp(v):
    a = np.maximum(np.abs(v), 2.0 ** -126)
    return 2.0 ** (np.floor(np.log2(a)) - 8)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32], ids=str)
def test_rmsnorm_dropout_forward(T, H, w_dtype):
    x, res, _, _, w = rms_case(T, H, T + H, w_dtype)
    p, seed, offset = 0.2, 123456789012345, 1 << 35
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, p, seed, offset)
    check_sum(h, x, p, seed, offset, res)
    assert torch.equal(h, R.dropout_fwd(x, p, seed, offset, residual=res))
    h64 = f64(h)
    r64 = 1 / np.sqrt((h64 * h64).mean(1) + float(np.float32(1e-6)))
    assert (np.abs(f64(rstd) - r64) <= 1e-6 * r64).all()   # rmsnorm_train_fwd's own bound
    y64 = h64 * r64[:, None] * f64(w)
    # rstd's error, two FP32 products, the rounding to bf16
    e = np.abs(y64) * (1e-6 + 2.0 ** -23)
    assert (np.abs(f64(y) - y64) <= e + half_ulp(np.abs(y64) + e)).all()
    assert N.rmsnorm_train_device_error(reset=True) == 0


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("with_dh", [False, True])
def test_rmsnorm_dropout_backward(T, H, with_dh):
    x, res, dy, dh, w = rms_case(T, H, T + H + 50, torch.float32 if with_dh else torch.bfloat16)
    dh = dh if with_dh else None
    p, seed, offset = 0.3, 42, 7
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, p, seed, offset)
    dx, dres, dw = R.rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, offset, dh=dh)
    # the norm's part is rmsnorm_bwd's, bit for bit
    dres0, dw0 = R.rmsnorm_bwd(dy, h, rstd, w, dh=dh)
    assert torch.equal(dres, dres0) and torch.equal(dw, dw0)
    h64, dy64, w64, r64 = f64(h), f64(dy), f64(w), f64(rstd)
    dx64, total, dw64 = OD.rmsnorm_bwd(h64, dy64, None if dh is None else f64(dh), r64, w64, p,
                                       seed, offset)
    # FP32 value of total: the roundings of g, xhat c, their difference and the scaling, and the
    # row sum's (at most ~32 deep) -- rmsnorm_train_bwd's allowance; then scale and its product
    xh, g = h64 * r64[:, None], dy64 * w64
    c = (g * xh).mean(1, keepdims=True)
    allow = r64[:, None] * (2.0 ** -20 * (np.abs(g) + np.abs(xh * c)) +
                            2.0 ** -18 * np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    if dh is not None:
        allow += 2.0 ** -23 * np.abs(f64(dh))
    assert (np.abs(f64(dres) - total) <= allow + half_ulp(np.abs(total) + allow)).all()
    k = OD.keep(h.numel(), p, seed, offset).reshape(h64.shape)
    e = OD.scale(p) * allow + np.abs(dx64) * 2.0 ** -23
    assert (np.abs(f64(dx) - dx64)[k] <= (e + half_ulp(np.abs(dx64) + e))[k]).all()
    assert not f64(dx)[~k].any()
    assert (np.abs(f64(dw) - dw64) <= 1e-4 + 1e-4 * np.abs(dw64)).all()
    # the other mode: the same dx and dres, dw within the budget
    dx1, dres1, dw1 = R.rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, offset, deterministic=False,
                                            dh=dh)
    assert torch.equal(dx, dx1) and torch.equal(dres, dres1)
    assert (np.abs(f64(dw1) - dw64) <= 1e-4 + 1e-4 * np.abs(dw64)).all()
    assert N.rmsnorm_train_device_error(reset=True) == 0


def test_rmsnorm_dropout_edges_of_p():
    x, res, dy, dh, w = rms_case(300, 256, 5, torch.float32)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, 0.0, 3)
    y0, rstd0, h0 = R.rmsnorm_fwd(x, w, residual=res)
    assert torch.equal(y, y0) and torch.equal(rstd, rstd0) and torch.equal(h, h0)
    dx, dres, _ = R.rmsnorm_dropout_bwd(dy, h, rstd, w, 0.0, 3, dh=dh)
    assert torch.equal(dx, dres)
    few = R.rmsnorm_dropout_bwd(dy[:9], h[:9], rstd[:9], w, 0.0, 3, dh=dh[:9])
    assert torch.equal(few[0], few[1])
    x[5] = float("nan")                           # everything is dropped, whatever it is
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, 1.0, 3)
    assert torch.equal(h, res)
    dx, dres, _ = R.rmsnorm_dropout_bwd(dy, h, rstd, w, 1.0, 3, dh=dh)
    assert not dx.any() and dres.any()


def test_rmsnorm_dropout_many_rows_a_cta():
    # rings that go round many times, and the non-deterministic mode's pool open
    T, H = 40000, 256
    x, res, dy, dh, w = rms_case(T, H, 6, torch.float32)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, 0.1, 17, 5)
    assert torch.equal(h, R.dropout_fwd(x, 0.1, 17, 5, residual=res))
    ref = R.rmsnorm_bwd(dy, h, rstd, w, dh=dh)
    for det in (True, False):
        dx, dres, dw = R.rmsnorm_dropout_bwd(dy, h, rstd, w, 0.1, 17, 5, deterministic=det,
                                             dh=dh)
        assert torch.equal(dres, ref[0])
        assert torch.equal(dx != 0, (R.dropout_bwd(torch.ones_like(dres), 0.1, 17, 5) != 0) &
                           (dres != 0))
    assert N.rmsnorm_train_device_error(reset=True) == 0


def test_rmsnorm_dropout_views():
    # the first heads of a wider buffer: the mask goes by the logical index, not the address
    T, nh, H = 37, 3, 256
    wide, wide_r = normal(1, T, 5 * H), normal(2, T, 5 * H)
    x, r = (b.view(T, 5, H)[:, :nh] for b in (wide, wide_r))
    w = 1 + 0.1 * normal(3, H, dtype=torch.float32)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, r, w, 0.4, 8)
    y1, rstd1, h1 = R.rmsnorm_dropout_fwd(x.contiguous(), r.contiguous(), w, 0.4, 8)
    assert torch.equal(h, h1) and torch.equal(y, y1) and torch.equal(rstd, rstd1)
    assert torch.equal(h, R.dropout_fwd(x.contiguous(), 0.4, 8, residual=r.contiguous()))
    dx, dres, dw = R.rmsnorm_dropout_bwd(y, h, rstd, w, 0.4, 8)
    flat = R.rmsnorm_dropout_bwd(y.view(-1, H), h.view(-1, H), rstd.view(-1), w, 0.4, 8)
    assert torch.equal(dx.view(-1, H), flat[0]) and torch.equal(dw, flat[2])


def test_rmsnorm_dropout_no_rows():
    w = torch.ones(64, device=DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, x, w, 0.5, 1)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dres, dw = R.rmsnorm_dropout_bwd(x, x, rstd, w, 0.5, 1)
    assert dx.shape == dres.shape == (0, 64) and not dw.any()


def test_rmsnorm_dropout_refusals():
    x = normal(1, 4, 64)
    w = torch.ones(64, device=DEV)
    with pytest.raises(ValueError, match="residual"):
        R.rmsnorm_dropout_fwd(x, x[:2], w, 0.5, 1)
    with pytest.raises(ValueError, match="w must"):
        R.rmsnorm_dropout_fwd(x, x, w[:32], 0.5, 1)
    rstd = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="dy"):
        R.rmsnorm_dropout_bwd(x.float(), x, rstd, w, 0.5, 1)
    with pytest.raises(ValueError, match="rstd"):
        R.rmsnorm_dropout_bwd(x, x, rstd[:2], w, 0.5, 1)
    with pytest.raises(ValueError, match="one device"):
        R.rmsnorm_dropout_bwd(x, x, rstd.cpu(), w, 0.5, 1)
    with pytest.raises(ValueError, match="contiguous"):
        R.rmsnorm_dropout_bwd(x[:, :32], x[:, :32], rstd, w[:32], 0.5, 1)


def test_rmsnorm_dropout_autograd():
    x, res, dy, dh, w = rms_case(70, 768, 8, torch.bfloat16)
    for t in (x, res, w):
        t.requires_grad_()
    y, h = R.rmsnorm_dropout_train(x, res, w, 0.1, 5, 1)
    (y.float() * dy.float()).sum().add((h.float() * dh.float()).sum()).backward()
    d = [t.detach() for t in (x, res, w)]
    y0, rstd0, h0 = R.rmsnorm_dropout_fwd(*d, 0.1, 5, 1)
    assert torch.equal(y, y0) and torch.equal(h, h0)
    dx, dres, dw = R.rmsnorm_dropout_bwd(dy, h0, rstd0, d[2], 0.1, 5, 1, dh=dh)
    assert torch.equal(x.grad, dx) and torch.equal(res.grad, dres)
    assert torch.equal(w.grad, dw.bfloat16())
    for t in (x, res, w):
        t.grad = None
    y, h = R.rmsnorm_dropout_train(x, res, w, 0.1, 5, 1)     # y unused: dh alone
    h.backward(dh)
    assert torch.equal(res.grad, dh) and torch.equal(x.grad, R.dropout_bwd(dh, 0.1, 5, 1))


def test_captured_step_draws_new_masks():
    T, H, p, seed = 300, 512, 0.25, 31
    x, res, dy, dh, w = rms_case(T, H, 12, torch.float32)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)

    def one_step():
        z = R.dropout_fwd(x, p, seed, 0, step=step)
        y, rstd, h = R.rmsnorm_dropout_fwd(z, res, w, p, seed, 1, step=step)
        out = (z, y, h) + R.rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, 1, step=step, dh=dh)
        step.add_(2)
        return out

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one_step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = one_step()
    masks = []
    for i in range(3):
        at = int(step)
        g.replay()
        torch.cuda.synchronize()
        assert int(step) == at + 2
        z = R.dropout_fwd(x, p, seed, at)
        y, rstd, h = R.rmsnorm_dropout_fwd(z, res, w, p, seed, at + 1)
        want = (z, y, h) + R.rmsnorm_dropout_bwd(dy, h, rstd, w, p, seed, at + 1, dh=dh)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        masks.append(z != 0)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])


def test_side_stream():
    x = normal(1, 4096, 1024)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x
        for i in range(8):                        # each call reads the one before it
            y = R.dropout_fwd(y, 0.1, 3, i)
    torch.cuda.current_stream().wait_stream(side)
    want = x
    for i in range(8):
        want = R.dropout_fwd(want, 0.1, 3, i)
    assert torch.equal(y, want)


def test_rmsnorm_dropout_elements_past_32_bits():
    T, H, p = (1 << 20) + 9, 4096, 0.5
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_()
    res = torch.empty_like(x).normal_()
    w = torch.ones(H, device=DEV)
    y, rstd, h = R.rmsnorm_dropout_fwd(x, res, w, p, 5, 6)
    assert torch.equal(h[-64:], R.dropout_fwd(x, p, 5, 6, residual=res)[-64:])
    k = torch.from_numpy(OD.keep(64 * H, p, 5, 6, (T - 64) * H)).to(DEV).view(64, H)
    del x, res
    dx, dres, _ = R.rmsnorm_dropout_bwd(y, h, rstd, w, p, 5, 6)
    assert torch.equal(dx[-64:] != 0, k & (dres[-64:] != 0))
