"""The AdamW step's square root where its two forms meet and where it has no value, to the bit against the oracle."""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, say
from oracle import adamw as oa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F = np.float32
HYPER = dict(lr=0.5, eps=1e-30, weight_decay=0.25, step=1)


def step(p, m, v, beta2=0.5):
    """(p, v) after a step with gradients of zero, here and from the oracle."""
    t = [torch.from_numpy(p.copy()).to(DEV)]
    st = g.adamw_init(t)
    st.m[:p.size].copy_(torch.from_numpy(m))
    st.v[:p.size].copy_(torch.from_numpy(v))
    g.adamw_step(t, [torch.zeros_like(t[0])], st, betas=(0.5, beta2), **HYPER)
    with np.errstate(invalid="ignore", divide="ignore"):
        rp, _, rv = oa.step_f32(p, np.zeros_like(p), m, v, beta1=0.5, beta2=beta2, **HYPER)[:3]
    return np32(t[0]), np32(st.v)[:p.size], rp, rv


def test_small_values_by_the_short_form():
    """Waves whose values all lie in [2^-96, 2^-60) after the step: every mantissa at both parities of the exponent, with
    residuals that are subnormal numbers in part."""
    r = np.random.default_rng(1)
    n = 1 << 24
    i = np.arange(n, dtype=np.uint32)
    # v halves; 127 - 95 = 32
    field = (r.integers(16, 34, n).astype(np.uint32) * 2 + (i >> 23)).astype(np.uint32)
    v = ((field << 23) | (i & 0x7FFFFF)).view(F)
    assert v.min() >= 2.0 ** -95 and v.max() < 2.0 ** -59
    p, pv, rp, rv = step(np.zeros(n, F), np.full(n, 2.0 ** -30, F), v)
    assert (pv == rv).all() and (p == rp).all(), int((p != rp).sum())


@pytest.mark.parametrize("beside", ["ordinary", "tiny", "infinite", "zero"])
@pytest.mark.parametrize("bad", [-1.0, -1e-8, -1e-20, -1e-25, -1e-40, float("-inf"), float("nan")])
def test_a_second_moment_without_a_root_shows(bad, beside):
    """A negative or NaN second moment (a state that something else broke) makes its parameter NaN whatever values its
    wave has beside it, and no other parameter changes."""
    r = np.random.default_rng(2)
    n = 2048
    p, m = r.normal(size=n).astype(F), r.normal(size=n).astype(F)
    v = (r.random(n) + 0.5).astype(F)
    if beside != "ordinary":
        v[5::64] = {"tiny": 2.0 ** -120, "infinite": np.inf, "zero": 0.0}[beside]
    at = np.arange(16, n, 512)
    v[at] = bad
    say("root", bad, beside)
    p, pv, rp, rv = step(p, m, v)
    assert np.isnan(rp[at]).all() and np.isnan(p[at]).all(), p[at]
    rest = np.ones(n, bool)
    rest[at] = False
    assert (p[rest] == rp[rest]).all() and (pv[rest] == rv[rest]).all()
