"""FP64 oracle of activations held in 8 bits (include/act8_train.h): the format in numpy, value by
value from its definition.  Shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
LOWEST, HIGHEST = -120, 127   # exponents


def row_bytes(h: int) -> int:
    pad = lambda n: (n + 15) // 16 * 16  # noqa: E731
    return pad(h) + pad((h + BLOCK - 1) // BLOCK)


def exponents(x):
    """x [R, H] float64: the exponent of each block, and whether it is all numbers, [R, blocks]."""
    r, h = x.shape
    n = (h + BLOCK - 1) // BLOCK
    full = np.zeros((r, n * BLOCK))
    full[:, :h] = x
    most = np.abs(full).reshape(r, n, BLOCK).max(2)
    ok = np.isfinite(most)
    m, k = np.frexp(np.where(ok, most, 1.0))
    e = k - 1                                  # most = 1.f * 2^e
    e = np.where(2 * m * 64 >= 127.5, e + 1, e)
    e = np.where((most > 0) & ok, e, LOWEST)
    return np.clip(e, LOWEST, HIGHEST), ok


def pack(x):
    """Packed rows of x [R, H] float64, as uint8 [R, row_bytes(H)]."""
    r, h = x.shape
    e, ok = exponents(x)
    col = np.arange(h) // BLOCK
    q = np.rint(np.where(ok[:, col], x, 0.0) * np.exp2(6.0 - e[:, col]))  # ties to even
    q = np.clip(q, -127, 127).astype(np.int8)
    out = np.zeros((r, row_bytes(h)), np.uint8)
    out[:, :h] = q.view(np.uint8)
    first = (h + 15) // 16 * 16
    out[:, first:first + e.shape[1]] = np.where(ok, e + 127, 255)
    return out


def unpack(p, h):
    """The values of packed rows, float64 [R, h]."""
    first = (h + 15) // 16 * 16
    col = np.arange(h) // BLOCK
    scale = p[:, first:first + (h + BLOCK - 1) // BLOCK].astype(np.int64)
    unit = np.where(scale == 255, np.nan, np.exp2(scale - 133.0))
    return np.ascontiguousarray(p[:, :h]).view(np.int8) * unit[:, col]


def held(x):
    return unpack(pack(x), x.shape[1])
