"""Pins of the 8-bit and AdamW oracles: closed forms, torch's optimizer and casts, bounds of the roundings."""
import numpy as np
import pytest
import torch

from oracle import adamw, e4m3, eightbit, layer as olayer
from oracle.layer import ExpertWeights


def test_codes_by_hand():
    codes, scale = eightbit.quantize_rows([[127.0, -127.0, 0.5, 1.5, -2.5, 0.0], [0.0] * 6, [2.0 ** -101] * 6])
    assert codes.tolist() == [[127, -127, 0, 2, -2, 0], [0] * 6, [0] * 6] and (np.abs(scale - 1) <= 2.0 ** -24).all()


def test_codes_are_nearest():
    x = np.random.default_rng(0).normal(size=(50, 64)).astype(np.float32)
    codes, scale = eightbit.quantize_rows(x)
    # half a step, and the roundings of scale, factor (two each) and product (2^-24 of up to 127 each)
    assert (np.abs(codes * scale[:, None].astype(np.float64) - x) <= (0.5 + 5 * 127 * 2.0 ** -24) * scale[:, None]).all()
    assert (np.abs(codes).max(axis=1) == 127).all()


def test_layer_against_the_float_layer():
    """Codes that stand for the weights exactly: what is left are the activations' roundings."""
    rng = np.random.default_rng(1)
    T, H, I, E, k = 9, 32, 48, 5, 2
    x = eightbit.bf16(rng.normal(size=(T, H)))
    logits = rng.normal(size=(T, E)).astype(np.float32)
    c13, c2 = rng.integers(-127, 128, (E, 2 * I, H)), rng.integers(-127, 128, (E, H, I))
    s13 = (0.01 * rng.random((E, 2 * I)) + 0.001).astype(np.float32)
    s2 = (0.01 * rng.random((E, H)) + 0.001).astype(np.float32)
    out = eightbit.forward(x, logits, c13.astype(np.int8), s13, c2.astype(np.int8), s2, k, num_valid_rows=15)
    ref = olayer.forward(x, logits, ExpertWeights(c13 * s13[..., None], c2 * s2[..., None]), k, 15)["out"]
    # x and h are off by half a step of amax / 127 each, 0.4% of the largest value, in a sum of 32 or 48
    assert np.abs(out - ref).max() / np.abs(ref).max() < 0.04
    assert (out[8] == 0).all()


@pytest.mark.parametrize("wd", [0.0, 0.1])
def test_formula_is_torchs(wd):
    torch.manual_seed(0)
    p = torch.randn(300, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=wd)
    q, m, v = p.detach().numpy().copy(), np.zeros(300), np.zeros(300)
    for t in range(1, 6):
        p.grad = torch.randn(300, dtype=torch.float64)
        q, m, v = adamw.formula(q, p.grad.numpy(), m, v, 1e-2, 0.8, 0.95, 1e-6, wd, t)
        opt.step()
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("schedule", [False, True])
def test_float32_steps_are_near_the_formula(schedule):
    rng = np.random.default_rng(2)
    p, g = rng.normal(size=1000).astype(np.float32), 1e-3 * rng.normal(size=1000).astype(np.float32)
    m, v = 1e-3 * rng.normal(size=1000).astype(np.float32), (1e-6 * rng.random(1000) + 1e-8).astype(np.float32)
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=7)
    sched = (1e-3, 1 - 0.9 ** 7, 1 - 0.99 ** 7) if schedule else None
    p1, m1, v1, _ = adamw.step_f32(p, 0.5 * g, m, v, grad_scale=1.0, schedule=sched, **hyper)
    p2, m2, v2 = adamw.formula(p, 0.5 * g.astype(np.float64), m, v, **hyper)
    u = 2.0 ** -24
    mags = 0.9 * np.abs(m) + 0.1 * 0.5 * np.abs(g)
    assert (np.abs(m1 - m2) <= 4 * u * mags).all() and (np.abs(v1 - v2) <= 5 * u * v2).all()
    # the update: m's error over the root, and 4 (v's half, root, factors) + 4 roundings of itself; the parameter 4
    root = np.sqrt(v2 / (1 - 0.99 ** 7))
    step = 1e-3 / (1 - 0.9 ** 7)
    assert (np.abs(p1 - p2) <= 4 * u * np.abs(p) + step * (4 * u * mags + 12 * u * np.abs(m2)) / root + u * np.abs(p2)).all()


def test_rounding_by_chance_is_exact_on_average():
    """Over all pieces a value's codes average to the value; exact codes stay."""
    piece = np.arange(65536)
    for x in (1.03, 300.7, 0.0131, 2.0 ** -9 * 0.3, 2.0 ** -6 * 1.01):
        q = adamw.by_chance(np.float32(x) + np.zeros(65536), piece, 3, -6, 0.5)
        step = 2.0 ** (max(np.frexp(x)[1] - 1, -6) - 3)
        assert abs(q.mean() - np.float32(x)) <= step / 65536 and len(set(q)) == 2
    vals = e4m3.decode(np.arange(127))
    for v in vals:
        assert (adamw.by_chance(np.full(3, v), np.array([0, 40000, 65535]), 3, -6, 0.5) == v).all()


def test_blocks():
    rng = np.random.default_rng(3)
    x = rng.normal(size=128).astype(np.float32)
    code, scale = adamw.code_block(x, None, False)
    one = np.float32(1)
    want = torch.from_numpy((x * (np.float32(448) * (one / np.abs(x).max()))).astype(np.float32)).to(torch.float8_e4m3fn)
    assert (code == want.view(torch.uint8).numpy()).all() and scale == np.abs(x).max() * (one / np.float32(448))
    assert (adamw.code_block(np.zeros(5, np.float32), None, True)[0] == 0).all()
    y = np.array([1.0, 1e-9, 0.0], np.float32)   # far below the block's largest: the least code, not zero
    for piece in (None, np.zeros(3)):
        assert adamw.code_block(y, piece, True)[0].tolist() == [126, 1, 0]
        assert adamw.code_block(y, piece, False)[0].tolist() == [126, 0, 0]
