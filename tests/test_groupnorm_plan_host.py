"""Group norm's plans over many samples, from the host functions alone."""
import math
import random

from rmsnorm_fwd_02_gb300 import _native as N


def shapes(seed, count):
    """(dtype, N, S, C, G) that the library takes: few and many samples, places and groups."""
    rng = random.Random(seed)
    while count:
        dtype = rng.randrange(3)
        ev = 4 if dtype == 1 else 8
        C = 8 * (rng.randint(1, 512) if rng.random() < 0.5 else int(2 ** rng.uniform(0, 9)))
        G = rng.choice([g for g in range(1, C + 1) if C % g == 0])
        if C // G * (ev // math.gcd(C // G, ev)) // ev > 512:
            continue
        S = rng.randint(1, 8) if rng.random() < 0.5 else int(2 ** rng.uniform(0, 16))
        most = min(2 ** 31 - 1, ((1 << 40) - 1) // (S * C))
        count -= 1
        yield dtype, most if rng.random() < 0.1 else min(most, int(2 ** rng.uniform(0, 21))), S, C, G


def test_workspace_stays_near_the_activation():
    # the worst of it: a place or two a sample, every channel in one slab, many samples
    worst = [(dtype, n, s, c, g) for dtype in (0, 1, 2) for n in (1, 300, 2500, 65536, 1 << 20)
             for s in (1, 2, 3, 4) for c, g in ((2048, 1), (4096, 1), (3000, 8), (4096, 32), (8, 1))
             if dtype != 1 or c // g <= 2048]
    for dtype, n, S, C, G in worst + list(shapes(5, 20000)):
        size = 4 if dtype == 1 else 2
        if S * C // G < 32:                       # (groups of a few values: their own sums count)
            continue
        for workspace in (N.groupnorm_train_fwd_workspace_bytes,
                          N.groupnorm_train_bwd_workspace_bytes):
            # the activation, an eighth of it for the groups' sums, one wave's column sums
            assert workspace(dtype, n, S, C, G) <= 1.125 * n * S * C * size + 2432 * 2 * C * 4


def test_units_and_pieces_fit_31_bits():
    for dtype, n, S, C, G in shapes(6, 20000):
        for bwd in (0, 1):
            p = N.groupnorm_train_launch_plan(dtype, n, S, C, G, bwd)
            if not p["on_chip"]:
                assert n * (C // p["channels"]) < 1 << 31
                assert p["units"] * p["chunks"] < 1 << 31


def test_units_of_few_elements_stay_on_chip():
    # which is what keeps the number of streamed units below 2^31
    for C in range(8, 4097, 8):
        for G in (g for g in range(1, C + 1) if C % g == 0):
            for dtype in (0, 1):
                ev = 4 if dtype == 1 else 8
                if C // G * (ev // math.gcd(C // G, ev)) // ev > 512:
                    continue
                for S in (1, 2, 3, 7, 32, 64, 128):
                    n = min(2 ** 31 - 1, ((1 << 40) - 1) // (S * C))
                    for bwd in (0, 1):
                        p = N.groupnorm_train_launch_plan(dtype, n, S, C, G, bwd)
                        assert p["on_chip"] or S * p["channels"] > 512
