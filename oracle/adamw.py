"""An AdamW step: the formula in float64, and in float32 one operation after the other with the
states' roundings, whose results are defined to the bit.

Test infrastructure only (see ``oracle/__init__``).  Loshchilov and Hutter, "Decoupled Weight Decay
Regularization" (ICLR 2019); the generator of ``dropout.py`` with counter word 2.
"""

from __future__ import annotations

import numpy as np

from . import dropout, e4m3
from .eightbit import bf16

F = np.float32
BLOCK = 128


def formula(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step):
    """float64 (p, m, v) after a step."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


def pieces(first: int, n: int, seed: int, offset: int) -> np.ndarray:
    """The 16-bit pieces of elements [first, first + n) of the state arrays."""
    out = np.empty(n, np.uint32)
    key = [seed & dropout.M32, (seed >> 32) & dropout.M32]
    words, last = None, None
    for i in range(n):
        at = first + i
        if at // 8 != last:
            last = at // 8
            ctr = (offset + last) & dropout.M64
            words = dropout.philox4x32([ctr & dropout.M32, ctr >> 32, 2, 0], key)
        out[i] = (words[at % 8 // 2] >> (16 * (at % 2))) & 0xFFFF
    return out


def by_chance(x, piece, mantissa: int, least: int, centre: float) -> np.ndarray:
    """float32 magnitudes rounded to `mantissa` bits (exponents from `least` on): down, or up where the
    remainder, as a share of a step, and (piece + centre) / 2^16 reach 1."""
    a = np.abs(np.asarray(x, np.float64))
    ex = np.maximum(np.frexp(a)[1] - 1, least)
    step = 2.0 ** (ex - mantissa)
    up = np.floor(a / step + (piece + centre) / 65536.0) * step
    return np.copysign(up, x)


def code_block(x, piece, least_one: bool):
    """-> (e4m3 codes, scale) of up to 128 float32 values."""
    amax = np.abs(x).max()
    if amax < F(2.0 ** -100):
        return np.zeros(x.shape, np.uint8), F(1.0)
    scale, inv = F(amax * (F(1.0) / F(448.0))), F(F(448.0) * (F(1.0) / amax))
    q = (x * inv).astype(F)
    if piece is None:
        code = e4m3.encode(q)
    else:
        # an e4m3 fraction of a step has 20 bits in float32: the sum that rounds takes 2^-6 for subnormals
        a = np.abs(q)
        small = a < F(2.0 ** -6)
        a = np.where(small, (a + F(2.0 ** -6)).astype(F), a)
        val = by_chance(a, piece, 3, -6, 0.5)
        val = np.minimum(np.where(small, val - 2.0 ** -6, val), 448.0)
        code = e4m3.encode(np.copysign(val, q).astype(F))
    if least_one:
        code = np.where((x > 0) & (code == 0), 1, code).astype(np.uint8)
    return code, scale


def step_f32(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0, schedule=None):
    """float32 (p, m, v, sqrt(v)) of flat float32 arrays, one rounding for each operation."""
    if schedule is None:
        decay, size = F(1.0 - lr * weight_decay), F(lr / (1.0 - beta1 ** step))
        root = F(1.0 / np.sqrt(1.0 - beta2 ** step))
    else:
        s = [F(t) for t in schedule]
        decay, size = F(F(1.0) - F(s[0] * F(weight_decay))), F(s[0] / s[1])
        root = F(F(1.0) / np.sqrt(s[2]))
    p, g, m, v = (np.asarray(t, F) for t in (p, g, m, v))
    g = g * F(grad_scale)
    m = m * F(beta1) + g * F(1.0 - beta1)
    v = v * F(beta2) + (g * g) * F(1.0 - beta2)
    u = np.sqrt(v)
    upd = m / (u * root + F(eps))
    return p * decay - upd * size, m, v, u
