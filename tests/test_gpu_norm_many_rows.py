"""Layer norm (forward, backward) of many rows: from 512 rows on a row has fewer waves and more chunks a lane, and a block
walks several rows with the next one's loads in flight.  Every row is different and compared with the
formula in 64 bits.

Tolerances are those of a row's sums: at most 32 terms in a lane, 6 additions in the wave, 4 over the
waves, each off by u = 2^-24 of the sum of magnitudes, and the few roundings of the formula: 128 u in all; a
rounding to bf16 adds 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from helpers import say
from oracle import norm as onorm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}

# (waves of a row, widths: one of whole 16-byte units and one that is not) for each layout of a row over
# waves and chunks of many rows
BF16 = [(1, 512, 509), (1, 1024, 1001), (2, 2048, 1531), (4, 4096, 2881), (8, 8192, 7169), (16, 16384, 12001),
        (16, 24576, 20001), (16, 32768, 32761)]
F32 = [(1, 256, 251), (1, 512, 509), (1, 768, 701), (1, 1024, 1021), (2, 1536, 1531), (2, 2048, 2047),
       (4, 2880, 2881), (4, 4096, 3585), (8, 6144, 5001), (8, 8192, 7169), (16, 12288, 10001), (16, 16384, 14001),
       (16, 20480, 17001), (16, 24576, 23001), (16, 28672, 26001), (16, 32768, 31001)]
CASES = [(torch.bfloat16, W, H) for W, *hs in BF16 for H in hs] + [(torch.float32, W, H) for W, *hs in F32 for H in hs]


def formula(x, w, b, eps, rms):
    """y, mean, rstd and the normalised rows in 64 bits, on the GPU."""
    x = x.double()
    mean = x.mean(1) if not rms else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    z = d * rstd[:, None]
    y = z if w is None else z * w.double()
    return (y if b is None else y + b.double()), mean, rstd, z


def check(T, H, dtype, wdt, bias, rms):
    import grouped_gemm_histogram_amd as g
    say(f"layer_norm T={T} H={H} {dtype} weight={wdt} bias={bias} rms={rms}")
    gen = torch.Generator(device=DEV).manual_seed(T * 131 + H)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)
    x = (rand(T, H) * (1.0 + rand(T, 1).abs()) + rand(T, 1)).to(dtype)      # each row its own offset and spread
    w = None if wdt is None else (0.2 * rand(H) + 1.0).to(wdt)
    b = rand(H).to(wdt or torch.float32) if bias else None
    y, stats = g.layer_norm(x, w, b, 1e-5, rms, return_stats=True)
    ref, mean, rstd, z = formula(x, w, b, 1e-5, rms)
    wa = 1.0 if w is None else w.double().abs()
    ba = 0.0 if b is None else b.double().abs()
    tol = 128 * U * (wa * (1 + z.abs()) + ba) + HALF[dtype] * ref.abs()
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert bool(((stats.rstd.double() - rstd).abs() <= 128 * U * rstd).all())
    if not rms:
        assert bool(((stats.mean.double() - mean).abs() <= 128 * U * x.double().abs().mean(1)).all())
    # the formula used here is the oracle's
    rows = [0, T // 2, T - 1]
    host = lambda t: None if t is None else t.double().cpu().numpy()
    want, om, orr = onorm.layer_norm(host(x[rows]), host(w), host(b), 1e-5, rms)
    np.testing.assert_allclose(host(ref[rows]), want, rtol=1e-11, atol=1e-11)
    np.testing.assert_allclose(host(rstd[rows]), orr, rtol=1e-12)
    if not rms:
        np.testing.assert_allclose(host(mean[rows]), om, rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("dtype,W,H", CASES)
def test_blocks_that_walk_rows(dtype, W, H):
    """4096 / W rows are in flight at a time: some blocks have three rows and some two."""
    check(2 * 4096 // W + 37, H, dtype, torch.float32, True, False)
    check(2 * 4096 // W + 37, H, dtype, torch.bfloat16, False, True)


@pytest.mark.parametrize("T", [511, 512, 513])
@pytest.mark.parametrize("H", [64, 2880, 2881, 7168, 12001])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_both_sides_of_few_rows(T, H, dtype):
    check(T, H, dtype, None, True, False)
    check(T, H, dtype, torch.float32, True, True)


# the layouts of the backward, which takes up to three chunks a lane of bf16 before a row has more waves
BWD = [(torch.bfloat16, W, H) for W, *hs in [
    (1, 512, 509), (1, 1024, 1001), (1, 1536, 1531), (2, 2048, 2047), (2, 2880, 2881), (4, 4096, 3585),
    (4, 6144, 5001), (8, 8192, 7169), (8, 12288, 10001), (16, 16384, 12500), (16, 24576, 20001),
    (16, 32768, 30001)] for H in hs] + [(torch.float32, W, H) for W, *hs in F32 for H in hs]


@pytest.mark.parametrize("dtype,W,H", BWD)
def test_backward_blocks_that_walk_rows(dtype, W, H):
    """256 blocks of 8 waves (16 for the widest) walk the rows; the statistics are the formula's."""
    import grouped_gemm_histogram_amd as g
    T = 2 * 256 * max(8 // W, 1) + 37
    for rms, wdt, bias in ((False, torch.float32, True), (True, torch.bfloat16, False)):
        say(f"layer_norm_backward T={T} H={H} {dtype} rms={rms} weight={wdt} bias={bias}")
        gen = torch.Generator(device=DEV).manual_seed(T * 131 + H)
        rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)
        x = (rand(T, H) * (1.0 + rand(T, 1).abs()) + rand(T, 1)).to(dtype)
        dy, w = rand(T, H).to(dtype), (0.2 * rand(H) + 1.0).to(wdt)
        _, mean, rstd, _ = formula(x, None, None, 1e-5, rms)
        stats = g.NormStats(None if rms else mean.float(), rstd.float())
        gr = g.layer_norm_backward(dy, x, stats, w, bias_grad=bias)
        r = stats.rstd.double()[:, None]
        xhat = (x.double() if rms else x.double() - stats.mean.double()[:, None]) * r
        gg = dy.double() * w.double()
        m1 = 0.0 if rms else gg.mean(1, keepdim=True)
        dx = r * (gg - m1 - xhat * (gg * xhat).mean(1, keepdim=True))
        a1, a2 = gg.abs().mean(1, keepdim=True), (gg * xhat).abs().mean(1, keepdim=True)
        tol = 128 * U * r * (gg.abs() + a1 + xhat.abs() * a2) + HALF[dtype] * dx.abs()
        assert bool(((gr.dx.double() - dx).abs() <= tol).all())
        # a column: its rows in a slot, the slots in a tree, 16 of the 256 partial rows a wave, 16 waves
        n = 64 + T / 128
        p = dy.double() * xhat
        assert bool(((gr.dweight.double() - p.sum(0)).abs() <= (n + 4) * U * p.abs().sum(0)).all())
        if bias:
            assert bool(((gr.dbias.double() - dy.double().sum(0)).abs() <= n * U * dy.double().abs().sum(0)).all())
