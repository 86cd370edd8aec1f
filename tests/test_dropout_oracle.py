"""Pins of the dropout oracle: the generator's published known answers, the definition's
edges, the mask's distribution, and its gradients against central differences."""
import numpy as np
import pytest

from oracle import dropout as OD


@pytest.mark.parametrize("counter,key,want", [
    # the known answers published with the generator, ten rounds
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_known_answers(counter, key, want):
    assert OD.philox(counter, key) == want


@pytest.mark.parametrize("seed,counter,first", [
    (0, 0, 0), ((1 << 64) - 1, (1 << 64) - 1, 0), (0x299F31D0A4093822, 0x0370734413198A2E, 8 * 12345),
    (7, 1 << 40, 8 * ((1 << 33) + 5)),
])
def test_numbers_follow_the_block_function(seed, counter, first):
    got = OD.numbers(41, seed, counter, first)
    for i in range(41):
        q = (first + i) // 8
        b = OD.philox([q & OD.LOW, q >> 32, counter & OD.LOW, counter >> 32],
                      [seed & OD.LOW, seed >> 32])
        j = (first + i) % 8
        assert got[i] == (b[j // 2] >> (16 * (j % 2))) & 0xFFFF


def test_threshold_and_scale():
    assert OD.threshold(0.0) == 0 and OD.scale(0.0) == 1.0
    assert OD.threshold(1.0) == 65536 and OD.scale(1.0) == 0.0
    assert OD.threshold(0.5) == 32768 and OD.scale(0.5) == 2.0
    assert OD.threshold(2.0 ** -18) == 0 and OD.threshold(2.0 ** -17) == 1
    assert OD.keep(1000, 0.0, 1, 2).all() and not OD.keep(1000, 1.0, 1, 2).any()


def test_mask_distribution():
    n = 1 << 20
    for p in (0.1, 0.5, 0.9):
        k = OD.keep(n, p, 1234, 0)
        q = 1 - OD.threshold(p) / 65536
        assert abs(k.mean() - q) < 5 * np.sqrt(q * (1 - q) / n)
        a = k.astype(float) - q          # neighbours, places of a block and blocks: independent
        for lag in (1, 2, 7, 8, 9, 4096):
            assert abs((a[:-lag] * a[lag:]).mean()) < 5 * q * (1 - q) / np.sqrt(n - lag)
    other = OD.keep(n, 0.5, 1234, 1)
    assert abs((other == OD.keep(n, 0.5, 1234, 0)).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)


def test_rmsnorm_dropout_gradient_against_differences():
    rng = np.random.default_rng(5)
    R, H, p, seed, ctr, eps = 3, 16, 0.4, 99, 7, 1e-3
    x, res, dy, dh = (rng.normal(size=(R, H)) for _ in range(4))
    w = 1 + 0.1 * rng.normal(size=H)

    def forward(x, res, w):
        h = OD.fwd(x, p, seed, ctr, res)
        rstd = 1 / np.sqrt((h * h).mean(1) + eps)
        return h, rstd, (dy * h * rstd[:, None] * w).sum() + (dh * h).sum()

    h, rstd, _ = forward(x, res, w)
    got = OD.rmsnorm_bwd(h, dy, dh, rstd, w, p, seed, ctr)
    step = 1e-5
    for i, (arg, grad) in enumerate(zip((x, res, w), got)):
        num = np.zeros_like(arg)
        for at in np.ndindex(arg.shape):
            args = [x.copy(), res.copy(), w.copy()]
            args[i][at] += step
            up = forward(*args)[2]
            args[i][at] -= 2 * step
            num[at] = (up - forward(*args)[2]) / (2 * step)
        # central differences: step^2 times a third derivative of order one, and 1e-16 / step
        assert np.abs(num - grad).max() < 1e-7
