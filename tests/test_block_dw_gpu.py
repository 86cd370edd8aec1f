"""The norms' dw and the gate's gradient of a block's boundary, and the dw of the norm that keeps 8
bits, over many rows: within the budget to which this library holds the dw of its norms, 1e-4 +
1e-4 |dw| of the 64-bit sum (include/rmsnorm_train.h, include/layernorm_train.h).

Why it holds, for values of both signs and size 1: an addition errs by 2^-25 (a third of that in
mean square: 0.29 ulp) of a partial sum of sqrt(k) after k rows.  n rows in one chain, of which R / n
are added exactly: sqrt(n R / 2) * 2^-24 * 0.4, at R = 65536 and n = 431 9e-5 rms and up to four times that
over the columns, past the budget where |dw| happens to be small.  In two levels of f and n / f rows
sqrt(f / n + 1 / f) of it, a third: 3e-5."""
import pytest
import torch

import rmsnorm_fwd_02_gb300 as R
from block_cases import DEV

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).bfloat16()


def column_sums(rows, f):
    """The 64-bit sum of f(rows i to j), in parts."""
    return sum(f(slice(i, i + 8192)).sum(0) for i in range(0, rows, 8192))


def within(got, want):
    far = ((got.double() - want).abs() / (1e-4 + 1e-4 * want.abs())).max().item()
    assert far <= 1, far


@pytest.mark.parametrize("rows,h", [(65536, 8192), (131072, 4096), (1000000, 512), (2000000, 256)])
def test_norms(rows, h):
    x, dy, w = normal(rows, rows, h), normal(rows + 1, rows, h), torch.ones(h, device=DEV)

    def exact(x, r):
        return column_sums(rows, lambda i: dy[i].double() * (x[i].double() * r[i].double()[:, None]))

    _, r, x8 = R.rmsnorm_act8_fwd(x, w)
    within(R.rmsnorm_act8_bwd(dy, x8, r, w)[1], exact(R.act8_unpack(x8, h), r))
    dw, want = R.rmsnorm_block_bwd(dy, None, x, r, None, w)[2], exact(x, r)
    within(dw, want)
    # the norm behind: S = sum of dh * xhat
    grads = R.rmsnorm_block_bwd(None, x, None, None, r, None, w, dh=dy)
    within(grads[3], want)
    # and a gate a sample: with a factor of one a sample's sum each, and their sum
    gate = torch.ones(2, h, device=DEV)
    grads = R.rmsnorm_block_bwd(None, x, None, None, r, None, w, gate, dh=dy)
    within(grads[3], want)
    half = rows // 2
    for n in range(2):
        i = slice(n * half, (n + 1) * half)
        within(grads[4][n], column_sums(half, lambda k: dy[i][k].double() *
                                        (x[i][k].double() * r[i][k].double()[:, None])))


@pytest.mark.parametrize("packed", [False, True])
def test_both_norms(packed):
    rows, h = 65536, 6144
    x, dy, w = normal(1, rows, h), normal(2, rows, h), torch.ones(h, device=DEV)
    _, hid, r2, r1, x8, h8 = R.rmsnorm_block_fwd(x, x, w, w, act8=True)
    kept = (x8, h8) if packed else (x, hid)
    grads = R.rmsnorm_block_bwd(dy, *kept, r2, r1, w, w)
    held = R.act8_unpack(h8, h) if packed else hid
    within(grads[2], column_sums(rows, lambda i: dy[i].double() * (held[i].double() *
                                                                   r2[i].double()[:, None])))
