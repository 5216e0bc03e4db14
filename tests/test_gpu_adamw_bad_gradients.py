"""What a gradient that is NaN, infinite or too large to be squared does to 8-bit states, in its step and in the next."""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, npu8
from oracle import e4m3

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F = np.float32
N, AT = 384, 200          # three blocks; the element in the middle one
BLOCK = slice(128, 256)


def run(bad, random, bits=8):
    """(parameters, m, sqrt(v) or v) before the steps, after one with `bad` at AT and after one without it, and the same
    of a run with a gradient of 0.01 there."""
    out = []
    for value in (bad, 0.01):
        gen = torch.Generator(device=DEV).manual_seed(1)
        p = [torch.randn(N, device=DEV, generator=gen)]
        gr = [0.01 * torch.randn(N, device=DEV, generator=gen)]
        gr[0][AT - 5] = 0.0                    # an element whose second moment stays zero
        gr[0][128] = 1.0                       # the block's largest
        st = g.adamw_init(p, bits=bits)
        rng = torch.tensor([7, 0], dtype=torch.int64, device=DEV) if random else None
        seen = []
        for step in (1, 2):
            now = gr[0].clone()
            if step == 1:
                now[AT] = value
            g.adamw_step(p, [now], st, lr=1e-2, step=step, weight_decay=0.1, rng=rng)
            if rng is not None:
                rng[1] += g.adamw_counters(p)
            values = lambda t, s: e4m3.decode(npu8(t)) if s is not None else np32(t)
            seen.append((np32(p[0]).copy(), values(st.m, st.m_scale).copy(), values(st.v, st.v_scale).copy(),
                         None if bits == 32 else np32(st.m_scale).copy(), None if bits == 32 else np32(st.v_scale).copy()))
        out.append(seen)
    return out


def others(a):
    return np.delete(a, AT)


@pytest.mark.parametrize("random", [False, True])
def test_nan_is_its_element_only(random):
    got, clean = run(float("nan"), random)
    for a, b in zip(got, clean):
        for x, y in zip(a[:3], b[:3]):
            assert np.isnan(x[AT]) and (others(x) == others(y)).all()
        assert (a[3] == b[3]).all() and (a[4] == b[4]).all()


@pytest.mark.parametrize("random", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinity_is_its_block_from_the_next_step_on(sign, random):
    got, clean = run(sign * float("inf"), random)
    (p1, m1, u1, sm, sv), (p2, m2, u2, _, _) = got
    assert np.isnan(p1[AT]) and (others(p1) == others(clean[0][0])).all()
    assert np.isinf(sm[1]) and np.isinf(sv[1]) and np.isfinite(sm[[0, 2]]).all() and np.isfinite(sv[[0, 2]]).all()
    assert np.isnan(m1[AT]) and np.isnan(u1[AT])
    assert np.isnan(p2[BLOCK]).all() and np.isnan(m2[BLOCK]).all()
    rest = np.ones(N, bool)
    rest[BLOCK] = False
    for a, b in ((p2, clean[1][0]), (m2, clean[1][1]), (u2, clean[1][2])):
        assert (a[rest] == b[rest]).all()


@pytest.mark.parametrize("random", [False, True])
def test_infinite_square_stops_its_block_from_the_next_step_on(random):
    """A gradient of 2^64 in f32: m stays finite, v does not."""
    got, clean = run(2.0 ** 64, random)
    (p1, m1, u1, sm, sv), (p2, _, _, _, _) = got
    assert (others(p1) == others(clean[0][0])).all()
    gen = torch.Generator(device=DEV).manual_seed(1)
    start = np32(torch.randn(N, device=DEV, generator=gen))
    decayed = lambda x: (x * F(1.0 - 1e-2 * 0.1)).astype(F)
    assert p1[AT] == decayed(start[AT])                       # m / infinity: nothing but the decay
    assert np.isfinite(sm).all() and np.isinf(sv[1]) and np.isfinite(sv[[0, 2]]).all()
    block = np.zeros(N, bool)
    block[BLOCK] = True
    none = np.zeros(N, bool)
    none[[AT, AT - 5]] = True                                 # the element, and one whose second moment is zero
    assert np.isnan(p2[none]).all()
    assert (p2[block & ~none] == decayed(p1[block & ~none])).all()
    assert (p2[~block] == clean[1][0][~block]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 2.0 ** 64])
def test_f32_states_keep_it_in_its_element(bad):
    got, clean = run(bad, False, bits=32)
    for a, b in zip(got, clean):
        for x, y in zip(a[:3], b[:3]):
            assert (others(x) == others(y)).all()
    assert np.isnan(got[1][0][AT]) or bad == 2.0 ** 64
