"""CPU pins of the oracle's norm, dropout and 4-bit weights against something other than itself."""
import numpy as np
import pytest
import torch

from oracle import dropout, fourbit, norm


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("affine", [False, True])
def test_norm_matches_autograd(rms, affine):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 11, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(11, generator=g, dtype=torch.float64, requires_grad=True) if affine else None
    b = torch.randn(11, generator=g, dtype=torch.float64, requires_grad=True) if affine else None
    dy = torch.randn(5, 11, generator=g, dtype=torch.float64)
    if rms:
        y = torch.nn.functional.rms_norm(x, (11,), w, 1e-3)
        y = y if b is None else y + b
    else:
        y = torch.nn.functional.layer_norm(x, (11,), w, b, 1e-3)
    y.backward(dy)
    np_ = lambda t: None if t is None else t.detach().numpy()
    got, mean, rstd = norm.layer_norm(np_(x), np_(w), np_(b), 1e-3, rms)
    np.testing.assert_allclose(got, np_(y), rtol=0, atol=1e-12)
    dx, dw, db = norm.layer_norm_backward(np_(dy), np_(x), mean, rstd, np_(w), rms)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=0, atol=1e-12)
    if affine:
        np.testing.assert_allclose(dw, w.grad.numpy(), rtol=0, atol=1e-12)
        np.testing.assert_allclose(db, b.grad.numpy(), rtol=0, atol=1e-12)


def test_norm_gradient_matches_differences():
    rng = np.random.default_rng(0)
    x, w, dy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    for rms in (False, True):
        y, mean, rstd = norm.layer_norm(x, w, None, 1e-5, rms)
        dx, _, _ = norm.layer_norm_backward(dy, x, mean, rstd, w, rms)
        h = 1e-6
        for i in np.ndindex(x.shape):
            e = np.zeros_like(x)
            e[i] = h
            up, down = (norm.layer_norm(x + s * e, w, None, 1e-5, rms)[0] for s in (1, -1))
            # central difference: error h^2 f''' / 6 + 2^-53 / h, both below 1e-8 here
            assert abs(((up - down) * dy).sum() / (2 * h) - dx[i]) < 1e-7


# known answers published with the generator's paper (its reference test vectors)
PHILOX_KAT = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


@pytest.mark.parametrize("counter,key,want", PHILOX_KAT)
def test_philox_known_answers(counter, key, want):
    assert tuple(dropout.philox4x32(counter, key)) == want


def test_dropout_mask_rate_and_offsets():
    n = 40000
    u = dropout.uniforms(n, 0x123456789ABCDEF0, 7)
    # the mean of n uniforms is within 5 standard deviations, 2^32 / sqrt(12 n) each
    assert abs(u.mean() - 2.0 ** 31) < 5 * 2.0 ** 32 / np.sqrt(12 * n)
    # the block after: a call that starts one counter later sees the same stream eight elements on
    np.testing.assert_array_equal(dropout.uniforms(64, 5, 12)[8:], dropout.uniforms(56, 5, 13))
    # counters wrap at 2^64
    np.testing.assert_array_equal(dropout.uniforms(16, 5, (1 << 64) - 1)[8:], dropout.uniforms(8, 5, 0))
    assert dropout.keep_mask(n, 1, 0, 0.0).all() and not dropout.keep_mask(n, 1, 0, 1.0).any()
    x = np.arange(24, dtype=np.float64) + 1
    out = dropout.dropout_add(x, 9, 2, 0.5, residual=-x)
    assert set(np.unique(out / x)) <= {-1.0, 1.0}


def test_fourbit_values():
    np.testing.assert_array_equal(fourbit.E2M1[:8], [0, 0.5, 1, 1.5, 2, 3, 4, 6])
    np.testing.assert_array_equal(fourbit.E2M1[8:], -fourbit.E2M1[:8])
    codes = np.array([[0x10, 0xF8]], np.uint8)
    np.testing.assert_array_equal(fourbit.unpack(codes), [[0, 1, 8, 15]])
    np.testing.assert_array_equal(fourbit.dequantize(codes, np.array([[0.5, 2.0]], np.float32)), [[-4, -3.5, 0, 14]])
    np.testing.assert_array_equal(fourbit.dequantize(codes, np.array([[128, 126]], np.uint8)), [[0, 1, 0, -3]])


@pytest.mark.parametrize("fmt,group", [("int4", 32), ("int4", 64), ("int4", 128), ("mxfp4", 32)])
def test_fourbit_quantize_error(fmt, group):
    rng = np.random.default_rng(1)
    w = rng.standard_normal((2, 3, 128)).astype(np.float32)
    w[0, 1] = 0.0
    codes, scales = fourbit.quantize(w, fmt, group)
    back = fourbit.dequantize(codes, scales)
    amax = np.repeat(np.abs(w.reshape(2, 3, -1, group)).max(-1), group, axis=-1)
    if fmt == "int4":    # half a step of amax / 7
        assert (np.abs(back - w) <= amax / 14 * (1 + 1e-6)).all()
    else:                # half the widest step, 2 of at most 6 where amax is 4 to 8 units; 8 saturates to 6
        assert (np.abs(back - w) <= amax / 4 + 1e-12).all()
    assert (back[0, 1] == 0).all()
