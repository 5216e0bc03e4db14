"""4-bit weights with group scales: what the codes stand for, and how weights are coded.

Test infrastructure only (see ``oracle/__init__``).  Codes are [E, N, K/2] bytes, the even channel
in the low nibble.  int4: (code - 8) * scale, float scales per group; mxfp4: e2m1(code) *
2^(scale - 127), one byte per 32 channels.
"""

from __future__ import annotations

import numpy as np


def e2m1(code: int) -> float:
    """Sign, two exponent bits (bias 1), one mantissa bit; exponent 0 is subnormal."""
    ex, man = (code >> 1) & 3, code & 1
    mag = man * 0.5 if ex == 0 else (1.0 + 0.5 * man) * 2.0 ** (ex - 1)
    return -mag if code & 8 else mag


E2M1 = np.array([e2m1(c) for c in range(16)])


def unpack(codes) -> np.ndarray:
    codes = np.asarray(codes, np.uint8)
    out = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.uint8)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def dequantize(codes, scales) -> np.ndarray:
    """float64 values [..., K] of codes [..., K/2] and scales [..., K/group] (uint8: mxfp4)."""
    c = unpack(codes)
    scales = np.asarray(scales)
    if scales.dtype == np.uint8:
        v, s = E2M1[c], np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    else:
        v, s = c.astype(np.float64) - 8.0, scales.astype(np.float64)
    return v * np.repeat(s, c.shape[-1] // scales.shape[-1], axis=-1)


def quantize(w, fmt: str, group: int):
    """-> (codes, scales), one group at a time from float32 weights [..., K]."""
    w = np.asarray(w, np.float32)
    flat = w.reshape(-1, group)
    code = np.empty(flat.shape, np.uint8)
    scales = np.empty(flat.shape[0], np.uint8 if fmt == "mxfp4" else np.float32)
    for i, g in enumerate(flat):
        amax = np.abs(g).max()
        if fmt == "int4":
            s = np.float32(amax / np.float32(7.0))
            s = s if s > 0 else np.float32(1.0)
            scales[i] = s
            code[i] = np.clip(np.rint(g / s), -8, 7).astype(np.int64) + 8
            continue
        ex = 0 if amax == 0 else int(np.clip(np.frexp(np.float64(amax))[1] - 1 - 2, -127, 127))
        scales[i] = ex + 127
        for j, v in enumerate(g.astype(np.float64) / 2.0 ** ex):
            # nearest of the eight magnitudes, the even code on a tie
            best = min(range(8), key=lambda c: (abs(abs(v) - E2M1[c]), c & 1))
            code[i, j] = best | (8 if np.signbit(v) else 0)
    code = code.reshape(w.shape)
    packed = (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)
    return packed, scales.reshape(w.shape[:-1] + (w.shape[-1] // group,))
