"""Layer norm of rows and its root-mean-square form, forward and backward, in float64.

Test infrastructure only (see ``oracle/__init__``).  The backward takes the statistics it is
given (the forward's, rounded as the caller keeps them), so it is the formula's value for them.
"""

from __future__ import annotations

import numpy as np


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    """-> (y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, mean, rstd, weight=None, rms: bool = False):
    """-> (dx, dweight, dbias)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xhat = (x if rms else x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    dx = g - xhat * (g * xhat).mean(axis=1, keepdims=True)
    if not rms:
        dx = dx - g.mean(axis=1, keepdims=True)
    return rstd * dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)
