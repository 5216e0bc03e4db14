"""Dropout from Philox4x32-10, element by element in Python integers.

Test infrastructure only (see ``oracle/__init__``).  The generator is the one of Salmon, Moraes,
Dror and Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3" (SC 2011).
"""

from __future__ import annotations

import numpy as np

M32 = (1 << 32) - 1
M64 = (1 << 64) - 1


def philox4x32(counter, key, rounds: int = 10):
    """Four counter words and two key words -> four words."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def uniforms(n: int, seed: int, offset: int) -> np.ndarray:
    """The 32-bit uniforms of elements 0..n-1, as uint64."""
    out = np.empty(n, np.uint64)
    key = [seed & M32, (seed >> 32) & M32]
    for b in range((n + 7) // 8):
        ctr = (offset + b) & M64
        hi = philox4x32([ctr & M32, ctr >> 32, 0, 0], key)
        lo = philox4x32([ctr & M32, ctr >> 32, 1, 0], key)
        for j in range(min(8, n - 8 * b)):
            sh = 16 * (j % 2)
            out[8 * b + j] = ((hi[j // 2] >> sh) & 0xFFFF) << 16 | ((lo[j // 2] >> sh) & 0xFFFF)
    return out


def keep_mask(n: int, seed: int, offset: int, p: float) -> np.ndarray:
    return uniforms(n, seed, offset) >= np.uint64(round(p * 2.0 ** 32))


def dropout_add(x, seed: int, offset: int, p: float, residual=None):
    x = np.asarray(x, np.float64)
    keep = keep_mask(x.size, seed, offset, p).reshape(x.shape)
    out = np.zeros(x.shape)
    if p < 1.0:
        out[keep] = x[keep] / (1.0 - p)
    return out if residual is None else out + np.asarray(residual, np.float64)
