"""8-bit integers with a scale for each row, and the layer on them.

Test infrastructure only (see ``oracle/__init__``).  The coding's decisions are taken in float32, as
its definition says; products and sums are in float64 (of codes, exact).
"""

from __future__ import annotations

import numpy as np

from . import routing

TINY = np.float32(2.0 ** -100)


def quantize_rows(x):
    """float32 rows [..., H] -> (int8 codes, float32 scales [...])."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=-1)
    none = amax < TINY
    safe = np.where(none, np.float32(1.0), amax)
    one = np.float32(1.0)
    scale = np.where(none, one, safe * (one / np.float32(127.0))).astype(np.float32)
    inv = np.where(none, np.float32(0.0), np.float32(127.0) * (one / safe)).astype(np.float32)
    return np.rint(x * inv[..., None]).astype(np.int8), scale


def grouped_gemm(a, a_scale, b, b_scale, offsets, rows, silu):
    """Permuted rows a [M, K] with their scales x b [E, N, K] -> float64 [M, N or N/2] (and, with silu, gate and up)."""
    n_out = b.shape[1] // 2 if silu else b.shape[1]
    out = np.zeros((rows, n_out))
    gate, up = np.zeros((rows, n_out)), np.zeros((rows, n_out))
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        acc = np.asarray(a[lo:hi], np.float64) @ np.asarray(b[e], np.float64).T
        acc = acc * np.asarray(a_scale[lo:hi], np.float64)[:, None] * np.asarray(b_scale[e], np.float64)[None]
        if not silu:
            out[lo:hi] = acc
            continue
        gate[lo:hi], up[lo:hi] = acc[:, :n_out], acc[:, n_out:]
        with np.errstate(over="ignore"):
            out[lo:hi] = gate[lo:hi] / (1.0 + np.exp(-gate[lo:hi])) * up[lo:hi]
    return (out, gate, up) if silu else out


def bf16(x):
    """float64 rounded to float32 and then to bf16 (to nearest, ties to even), as float32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def forward(x, logits, w13, w13_scale, w2, w2_scale, k, num_valid_rows=-1, renormalize=True):
    """The layer: token rows and h (rounded to bf16) quantised, y rounded to bf16, the combine in float64."""
    E = w13.shape[0]
    ids, w = routing.route_topk(logits, k, num_valid_rows, renormalize)
    off, order, pos = routing.build_offsets(ids.reshape(-1), E)
    R = ids.size
    xq, xs = quantize_rows(x)
    tok = np.asarray(order) // k
    h, _, _ = grouped_gemm(xq[tok], xs[tok], w13, w13_scale, off, R, True)
    hq, hs = quantize_rows(bf16(h))
    y = bf16(grouped_gemm(hq, hs, w2, w2_scale, off, R, False)).astype(np.float64)
    T = x.shape[0]
    pos = np.asarray(pos).reshape(T, k)
    valid = pos < off[E]
    return (y[pos] * np.where(valid, w.reshape(T, k), 0.0)[..., None]).sum(axis=1)
