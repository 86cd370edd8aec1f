"""FP64 oracle of the dropout entry points (include/dropout_train.h): the Philox4x32-10 block
function (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC
2011) in Python integers and in numpy, the keep mask, and the operators in double precision.
Shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
LOW = 0xFFFFFFFF


def philox(counter, key, rounds=10):
    """One block in Python integers: four 32-bit words."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = M0 * c[0], M1 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & LOW, (p0 >> 32) ^ c[3] ^ k[1], p0 & LOW]
        k = [(k[0] + W0) & LOW, (k[1] + W1) & LOW]
    return c


def threshold(p: float) -> int:
    return int(np.floor(65536 * p + 0.5))


def scale(p: float) -> float:
    t = threshold(p)
    return 65536 / (65536 - t) if t < 65536 else 0.0


def numbers(n, seed, counter, first=0):
    """The 16-bit numbers of elements [first, first + n) (first a multiple of 8); counter is
    offset + step."""
    q = np.arange(first // 8, first // 8 + (n + 7) // 8, dtype=np.uint64)
    low = np.uint64(LOW)
    s = np.uint64(32)
    counter %= 1 << 64
    c = [q & low, q >> s, np.full_like(q, counter & LOW), np.full_like(q, counter >> 32)]
    k = [seed & LOW, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(M0), c[2] * np.uint64(M1)   # below 2^64
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k[0]), p1 & low,
             (p0 >> s) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + W0) & LOW, (k[1] + W1) & LOW]
    out = np.empty((q.size, 8), dtype=np.int64)
    for i in range(4):
        out[:, 2 * i] = c[i] & np.uint64(0xFFFF)
        out[:, 2 * i + 1] = c[i] >> np.uint64(16)
    return out.reshape(-1)[:n]


def keep(n, p, seed, counter, first=0):
    return numbers(n, seed, counter, first) >= threshold(p)


def fwd(x, p, seed, counter, residual=None):
    """x (float64, any shape): [residual +] keep * x * scale; a dropped x contributes 0."""
    k = keep(x.size, p, seed, counter).reshape(x.shape)
    y = np.where(k, x * scale(p), 0.0)
    return y if residual is None else y + residual


def rmsnorm_bwd(h, dy, dh, rstd, w, p, seed, counter):
    """Gradients of sum(dy * y) + sum(dh * h) with y = h * rstd(h) * w and h = residual +
    dropout(x), at the given rstd: (dx, dresidual, dw); h, dy, dh [R, H]."""
    xhat, g = h * rstd[:, None], dy * w
    total = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    if dh is not None:
        total = total + dh
    k = keep(h.size, p, seed, counter).reshape(h.shape)
    return np.where(k, total * scale(p), 0.0), total, (dy * xhat).sum(0)
