"""The backward of a block's boundary over so many rows that its column sums have two levels: each
build, in both activation types.

Rows are independent, so dx and dresidual have to be, bit for bit, those of calls on fewer rows (whose
builds test_block_gpu.py and test_block_builds_gpu.py hold to the oracle).  The sums are held to
those in 64 bits.  An addition errs by at most U of what it forms, so a sum of n rows in runs of f by
f + ceil(n / f) additions one after another, and at most 9 behind them (rows side by side, the last
level, the join), each of at most the sum of magnitudes; a term has two roundings of its own, and t
those of block_cases.check_bwd."""
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from block_builds import NO_GATE, NO_POST, NO_PRE, ONE, additions
from block_cases import DEV, SUM, U
from rmsnorm_fwd_02_gb300 import _native as N

pytestmark = pytest.mark.gpu

# 3 samples of as many rows as leave a thread's lane more than 64 in every form
LONG = [(950400, 8), (950400, 40), (950400, 96), (158400, 768), (59400, 1792), (59400, 2048),
        (39600, 2304), (19800, 7000), (19800, 8192)]
PART = 3300                  # rows of a call without a second level, a divisor of a sample


def normal(seed, *shape, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def sums64(dy, dh, x, h, r2, r1, w_pre):
    """For each of three samples the sums in 64 bits: dw_pre and its magnitudes, S and its, and S's
    error by t's."""
    out = [torch.zeros(5, (dh if dy is None else dy).shape[1], dtype=torch.float64, device=DEV)
           for _ in range(3)]
    rows = len(dh if dy is None else dy)
    for i in range(0, rows, PART):
        s = out[i * 3 // rows]
        i = slice(i, i + PART)
        t, et = 0, 0
        if dy is not None:
            hh, g = h[i].double() * r2[i].double()[:, None], dy[i].double() * w_pre.double()
            c, mag = (g * hh).mean(1, keepdim=True), (g * hh).abs().mean(1, keepdim=True)
            r = r2[i].double()[:, None]
            t = r * (g - hh * c)
            et = r * (4 * U * g.abs() + hh.abs() * (SUM * mag + 6 * U * c.abs()))
            s[0] += (dy[i].double() * hh).sum(0)
            s[1] += (dy[i].double() * hh).abs().sum(0)
        if dh is not None:
            t = t + dh[i].double()
            et = et + 2 * U * dh[i].double().abs()
        if x is not None:
            et = et + 2 * U * t.abs()
            xh = x[i].double() * (1 if r1 is None else r1[i].double()[:, None])
            s[2] += (t * xh).sum(0)
            s[3] += (t * xh).abs().sum(0)
            s[4] += (et * xh.abs()).sum(0)
    return out


def close(got, want, err, what):
    err = err + U * (want.abs() + err)
    assert ((got.double() - want).abs() <= err).all(), (what, ((got.double() - want).abs() / err).max())


def parts(f, n):
    """f on every PART rows, its first two results put together."""
    out = [f(slice(i, i + PART)) for i in range(0, n, PART)]
    return [torch.cat([o[k] for o in out]) for k in range(2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows,h", LONG)
def test_long_runs(rows, h, dtype):
    x, hid, dy, dh = (normal(h + k, rows, h, dtype=dtype) for k in range(4))
    x8, h8 = R.act8_pack(x), R.act8_pack(hid)
    r1, r2 = (0.5 + torch.rand(rows, device=DEV) for _ in range(2))
    w_pre, w_post = (1 + 0.1 * normal(h + k, h, dtype=torch.float32) for k in (5, 6))
    gates = normal(h + 7, 3, h, dtype=torch.float32)
    b, a = 0.75, 0.875
    for packed in (False, True):
        kx, kh = (x8, h8) if packed else (x, hid)
        vx, vh = (R.act8_unpack(t, h, torch.float32) if packed else t for t in (kx, kh))
        for pre, post, gate, grads in ((1, 1, "sample", 2), (1, 1, "row", 1), (1, 0, "sample", 2),
                                       (1, 0, "row", 1), (1, 0, None, 2), (1, 0, None, 1),
                                       (0, 1, "sample", 2)):
            gate_n = {"sample": gates, "row": gates[1], None: None}[gate]
            d_y, d_h = dy if pre else None, dh if grads == 2 else None
            args = dict(w_pre=w_pre if pre else None, w_post=w_post if post else None, scale=b,
                        residual_scale=a)
            flags = (not post) * NO_POST | (not pre) * NO_PRE | (gate is None) * NO_GATE | \
                (d_h is None) * ONE
            n = 3 if gate == "sample" else 1
            p = N.rmsnorm_block_train_launch_plan(rows, h, n, 1, packed, flags)
            reads_x = post or gate
            got = R.rmsnorm_block_bwd(d_y, kx if reads_x else None, kh if pre else None, r2, r1,
                                      gate=gate_n, dh=d_h, **args)

            def part(i, gate=gate, kx=kx, kh=kh, d_y=d_y, d_h=d_h, args=args, reads_x=reads_x):
                g = {"sample": gates[i.start * 3 // rows], "row": gates[1], None: None}[gate]
                return R.rmsnorm_block_bwd(None if d_y is None else d_y[i], kx[i] if reads_x else None,
                                           kh[i], r2[i], r1[i], gate=g,
                                           dh=None if d_h is None else d_h[i], **args)
            few = N.rmsnorm_block_train_launch_plan(PART, h, 1, 1, packed, flags)
            if (few["vectors"], few["row_threads"]) == (p["vectors"], p["row_threads"]):
                for k, want in enumerate(parts(part, rows)):
                    assert torch.equal(got[k], want), (pre, post, gate, grads, packed, k)
            sums = sums64(d_y, d_h, vx if reads_x else None, vh, r2, r1 if post else None, w_pre)
            c = 2 * U + additions(p, rows) * U
            total = sum(sums)
            if pre:
                close(got[2], total[0], c * total[1], "dw_pre")
            if gate is not None:
                one = w_post.double() if post else torch.ones_like(total[0])
                for k, s in enumerate(sums if n == 3 else [total]):
                    err = abs(b) * one.abs() * (s[4] + c * s[3] + 3 * U * s[2].abs())
                    close(got[4][k] if n == 3 else got[4], b * one * s[2], err, "dgate")
            if post:
                g = gates.double() if n == 3 else gates[1].double()[None]
                per = sums if n == 3 else [total]
                want = b * sum(g[k] * s[2] for k, s in enumerate(per))
                err = abs(b) * sum(g[k].abs() * (s[4] + c * s[3] + 4 * U * s[2].abs())
                                   for k, s in enumerate(per))
                close(got[3], want, err, "dw_post")


@pytest.mark.parametrize("rows,h", LONG[::2])
def test_the_eight_bit_norm_is_the_block_of_one_norm(rows, h):
    """Its backward is the same kernel's, with or without dh."""
    dy, dh = (normal(h + k, rows, h, dtype=torch.bfloat16) for k in (2, 3))
    h8 = R.act8_pack(normal(h, rows, h, dtype=torch.bfloat16))
    r, w = 0.5 + torch.rand(rows, device=DEV), 1 + 0.1 * normal(h, h, dtype=torch.float32)
    for d in (None, dh):
        dx, dw = R.rmsnorm_act8_bwd(dy, h8, r, w, dh=d)
        got = R.rmsnorm_block_bwd(dy, None, h8, r, None, w, dh=d)
        assert torch.equal(dx, got[1]) and torch.equal(dw, got[2])


def test_no_wait_gave_up():
    assert N.rmsnorm_block_train_device_error() == 0
