"""The layer for few tokens where its routing takes two experts a lane (65 to 128 experts), and its second kernel in
both widths with tens of routed experts; oracle and tolerances of test_gpu_decode."""
import numpy as np
import pytest

from helpers import np32, say
from oracle import routing
from test_gpu_decode import Case, FORMATS, UNIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k,valid,renormalize", [(16, 128, 8, 101, True), (16, 65, 4, -1, True), (5, 100, 16, 71, False),
                                                     (1, 128, 1, -1, False)])
def test_two_experts_a_lane(fmt, T, E, k, valid, renormalize):
    H = I = max(UNIT[fmt], 128)
    say("routing", fmt, T, E, k, valid, renormalize)
    got, ref = Case(fmt, T, H, I, E, k, seed=E + T).check(valid, renormalize)
    assert (np32(got)[np.abs(ref).sum(axis=1) == 0] == 0).all()


@pytest.mark.parametrize("E", [65, 100, 128])
def test_ties_between_a_lanes_experts(E):
    """Equal logits 64 experts apart, in one lane, and in neighbouring ones: the lower expert first."""
    c = Case("bf16", 16, 64, 64, E, 6, seed=E)
    c.logits[:8, 64:] = c.logits[:8, :E - 64]
    c.logits[8:] = np.round(c.logits[8:])              # many equal ones
    c.logits[10] = 0.0
    c.logits[11] = -0.0
    c.logits[11, ::2] = 0.0
    ids, _ = routing.route_topk(c.logits, 6)
    assert (np.asarray(ids).reshape(16, 6)[[10, 11]] == np.arange(6)).all()
    c.check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("wide", [False, True])
def test_tens_of_routed_experts_in_both_widths(fmt, wide):
    """16 tokens on 4 of 40 experts: more pairs of experts than waves, with 8 waves a workgroup (H above 2048) and 16."""
    H = 2176 if wide else 384
    I = max(UNIT[fmt], 128)
    say("experts", fmt, H)
    Case(fmt, 16, H, I, 40, 4, seed=21).check(valid=61)
