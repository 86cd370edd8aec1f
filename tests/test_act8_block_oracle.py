"""Pins of the oracles of 8-bit activations and of a block's boundary: the format's definition value
by value and its error bound, and the gradients against central differences."""
import numpy as np
import pytest

from oracle import act8 as OA
from oracle import block as OB


def brute(block):
    """A block's held values from the definition, an exponent after another."""
    m = max(abs(v) for v in block)
    if not np.isfinite(m):
        return [np.nan] * len(block)
    e = -120
    while e < 127 and m * 2.0 ** (6 - e) >= 127.5:
        e += 1
    out = []
    for v in block:
        q = round(v * 2.0 ** (6 - e))          # Python rounds ties to even
        out.append(max(-127, min(127, q)) * 2.0 ** (e - 6))
    return out


@pytest.mark.parametrize("h", [1, 7, 31, 32, 33, 64, 250])
def test_format(h):
    rng = np.random.default_rng(h)
    x = rng.normal(size=(6, h)) * np.exp2(rng.integers(-60, 60, size=(6, 1)).astype(float))
    x[1] = 0.0
    x[2] = np.exp2(-130.0) * rng.normal(size=h)
    x[3] = 127.5 / 64                      # rounds to 128 at 2^0: takes the next exponent
    x[4] = np.nextafter(127.5 / 64, 0)
    x[5, 0] = 1.9999 * 2.0 ** 127
    got = OA.held(x)
    for r in range(6):
        for b in range(0, h, 32):
            assert np.array_equal(got[r, b:b + 32], brute(list(x[r, b:b + 32])))
    assert OA.pack(x).shape == (6, OA.row_bytes(h)) and OA.row_bytes(h) % 16 == 0


def test_non_numbers_stay_in_their_block():
    x = np.ones((2, 70))
    x[0, 40], x[1, 69] = np.inf, np.nan
    got = OA.held(x)
    assert np.isnan(got[0, 32:64]).all() and np.isnan(got[1, 64:]).all()
    assert np.array_equal(got[0, :32], x[0, :32]) and np.array_equal(got[1, :64], x[1, :64])
    assert not OA.pack(x)[0, 32:64].any()


def test_error_is_at_most_a_127th_of_the_block():
    x = np.random.default_rng(0).normal(size=(500, 96))
    err = np.abs(OA.held(x) - x).reshape(500, 3, 32).max(2)
    assert (err <= np.abs(x).reshape(500, 3, 32).max(2) / 127).all()
    # 7 significant bits: BF16 holds them all
    m, _ = np.frexp(OA.held(x))
    assert np.array_equal(m * 128, np.rint(m * 128))


@pytest.mark.parametrize("post,pre,n", [(True, True, 0), (True, True, 1), (True, True, 3),
                                        (False, True, 0), (False, True, 3), (True, False, 1)])
def test_gradients_against_differences(post, pre, n):
    rng = np.random.default_rng(7)
    R, H, eps, a, b = 6, 8, 1e-3, 0.8, 0.6
    args = dict(x=rng.normal(size=(R, H)), residual=rng.normal(size=(R, H)))
    args["w_pre"] = 1 + 0.1 * rng.normal(size=H) if pre else None
    args["w_post"] = 1 + 0.1 * rng.normal(size=H) if post else None
    args["gate"] = rng.normal(size=(n, H)) if n else None
    dy, dh = rng.normal(size=(2, R, H))

    def loss(kw):
        y, h, r2, r1 = OB.fwd(**kw, scale=b, residual_scale=a, eps=eps)
        return (0.0 if y is None else (dy * y).sum()) + (dh * h).sum(), (h, r2, r1)

    _, (h, r2, r1) = loss(args)
    dx, dres, dw_pre, dw_post, dgate, _ = OB.bwd(
        dy if pre else None, dh, args["x"], h, r2, r1, args["w_pre"], args["w_post"],
        args["gate"], b, a)
    grads = dict(x=dx, residual=dres, w_pre=dw_pre, w_post=dw_post, gate=dgate)
    step = 1e-5
    for name, value in args.items():
        if value is None:
            assert grads[name] is None
            continue
        num = np.zeros_like(value)
        for at in np.ndindex(value.shape):
            up, down = value.copy(), value.copy()
            up[at] += step
            down[at] -= step
            num[at] = (loss({**args, name: up})[0] - loss({**args, name: down})[0]) / (2 * step)
        # central differences: step^2 times a third derivative of order ten, and 1e-15 / step
        assert np.abs(num - grads[name]).max() < 1e-7, name
