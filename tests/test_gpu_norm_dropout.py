"""Layer norm (forward, backward) and dropout on the GPU against the float64 oracle.

Tolerances.  u = 2^-24 is half a step of f32.  A row's sums have at most 64 terms in a lane, 6 in
the wave and 16 over the waves, so a sum is off by at most 86 u times the sum of magnitudes;
128 u covers that with the few further roundings of the formula.  A rounding to bf16 adds 2^-8
of the value.
"""
import numpy as np
import pytest
import torch

from helpers import say
from oracle import dropout as odrop, norm as onorm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def host(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def rand(seed, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale + shift).to(dtype).to(DEV)


# widths on both sides of every step of waves per row and chunks per lane, odd ones among them
WIDTHS = [1, 7, 64, 255, 513, 1024, 1531, 2048, 2880, 2881, 4095, 7168, 8200, 16384, 20001, 32768]


def norm_reference(x, w, b, eps, rms):
    y, mean, rstd = onorm.layer_norm(host(x), host(w), host(b), eps, rms)
    z = (host(x) - mean[:, None]) * rstd[:, None]
    wa = 1.0 if w is None else np.abs(host(w))
    ba = 0.0 if b is None else np.abs(host(b))
    tol = 128 * U * (wa * (1 + np.abs(z)) + ba) + HALF[x.dtype] * np.abs(y)
    return y, mean, rstd, tol


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm(H, rms, dtype):
    import grouped_gemm_histogram_amd as g
    for T, wdt, bias in ((1, torch.float32, True), (5, torch.bfloat16, False), (37, None, False)):
        say(f"layer_norm T={T} H={H} {dtype} rms={rms} weight={wdt} bias={bias}")
        x = rand(H + T, T, H, dtype=dtype, scale=2.0, shift=0.5)
        w = None if wdt is None else rand(1, H, dtype=wdt, scale=0.2, shift=1.0)
        b = rand(2, H, dtype=wdt) if bias else None
        y, stats = g.layer_norm(x, w, b, 1e-5, rms, return_stats=True)
        ref, mean, rstd, tol = norm_reference(x, w, b, 1e-5, rms)
        assert y.dtype == dtype and (np.abs(host(y) - ref) <= tol).all()
        assert (np.abs(host(stats.rstd) - rstd) <= 128 * U * rstd).all()
        if rms:
            assert stats.mean is None
        else:
            assert (np.abs(host(stats.mean) - mean) <= 128 * U * np.abs(host(x)).mean(1)).all()
        assert torch.equal(g.layer_norm(x, w, b, 1e-5, rms), y)


def test_layer_norm_far_from_zero_constant_and_special_rows():
    import grouped_gemm_histogram_amd as g
    H = 2880
    x = rand(0, 6, H)
    x[0] += 4096.0                       # spread far below the offset
    x[1] = 3.0                           # constant: variance 0, y = bias
    x[2] = 1e17 * x[2]                   # the sum of squares near the end of f32's range
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    say("layer_norm special rows")
    b = rand(3, H)
    y, stats = g.layer_norm(x, None, b, 1e-5, return_stats=True)
    ref, mean, rstd, tol = norm_reference(x[[0, 1, 2, 5]], None, b, 1e-5, False)
    assert (np.abs(host(y)[[0, 1, 2, 5]] - ref) <= tol).all()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.isnan(stats.rstd[3]) and torch.isnan(stats.rstd[4])
    z = g.layer_norm(torch.zeros(3, H, device=DEV), rms=True, eps=1e-5)
    assert (z == 0).all()


@pytest.mark.parametrize("H", [2880, 7168, 20001])
def test_layer_norm_same_rows_same_bits(H):
    """Many rows over several waves each: a row's result depends on the row alone."""
    import grouped_gemm_histogram_amd as g
    x = rand(9, 1, H, dtype=torch.bfloat16, shift=1.0).repeat(12000, 1)
    say(f"layer_norm same rows H={H}")
    y, stats = g.layer_norm(x, return_stats=True)
    assert (y == y[0]).all() and (stats.mean == stats.mean[0]).all() and (stats.rstd == stats.rstd[0]).all()
    dx = g.layer_norm_backward(y, x, stats).dx
    assert (dx == dx[0]).all()


def test_layer_norm_in_place_no_rows_and_refusals():
    import grouped_gemm_histogram_amd as g
    for H in (2880, 2881):
        x = rand(4, 300, H, dtype=torch.bfloat16)
        want = g.layer_norm(x, rms=True)
        assert g.layer_norm(x, rms=True, out=x) is x and torch.equal(x, want)
    empty = torch.empty(0, 64, device=DEV)
    y, stats = g.layer_norm(empty, return_stats=True)
    assert y.shape == (0, 64) and stats.rstd.shape == (0,)
    w = torch.ones(64, device=DEV)
    gr = g.layer_norm_backward(empty, empty, stats, w, bias_grad=True)
    assert (gr.dweight == 0).all() and (gr.dbias == 0).all() and gr.dx.shape == (0, 64)
    x = rand(5, 4, 64)
    with pytest.raises(ValueError, match="shape"):
        g.layer_norm(x, torch.ones(63, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        g.layer_norm(rand(5, 64, 4).t())
    with pytest.raises(ValueError, match="dtype"):
        g.layer_norm(x, torch.ones(64, device=DEV), torch.ones(64, device=DEV, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="dtype"):
        g.layer_norm(x.half())
    with pytest.raises(RuntimeError, match="MOE_ERR_UNSUPPORTED"):
        g.layer_norm(torch.zeros(1, 32769, device=DEV))
    with pytest.raises(RuntimeError, match="eps"):
        g.layer_norm(x, eps=-1.0)


def backward_reference(dy, x, stats, w, rms):
    mean, rstd = host(stats.mean), host(stats.rstd)
    dx, dw, db = onorm.layer_norm_backward(host(dy), host(x), mean, rstd, host(w), rms)
    xhat = (host(x) - (0 if rms else mean[:, None])) * rstd[:, None]
    gg = np.abs(host(dy) * (1.0 if w is None else host(w)))
    mg, mx = gg.mean(1, keepdims=True), (gg * np.abs(xhat)).mean(1, keepdims=True)
    tol = 128 * U * rstd[:, None] * (gg + mg + np.abs(xhat) * mx) + HALF[x.dtype] * np.abs(dx)
    # a column's sum: at most 64 + T / 128 additions in a row slot, a wave and a block
    n = 64 + x.shape[0] / 128
    adw, adb = (np.abs(host(dy) * xhat)).sum(0), np.abs(host(dy)).sum(0)
    return dx, dw, db, tol, (n + 4) * U * adw, n * U * adb


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer_norm_backward(H, rms, dtype):
    import grouped_gemm_histogram_amd as g
    for T, wdt, bias, gdt in ((1, torch.float32, True, torch.float32), (6, None, True, torch.bfloat16),
                              (1301 if H <= 2881 else 301, torch.bfloat16, False, torch.float32)):
        say(f"layer_norm_backward T={T} H={H} {dtype} rms={rms} weight={wdt} bias={bias} grads {gdt}")
        x = rand(H + T, T, H, dtype=dtype, shift=0.25)
        dy = rand(H + T + 1, T, H, dtype=dtype)
        w = None if wdt is None else rand(1, H, dtype=wdt, scale=0.2, shift=1.0)
        _, stats = g.layer_norm(x, w, None, 1e-5, rms, return_stats=True)
        gr = g.layer_norm_backward(dy, x, stats, w, bias_grad=bias, grad_dtype=gdt)
        dx, dw, db, tol, tw, tb = backward_reference(dy, x, stats, w, rms)
        assert (np.abs(host(gr.dx) - dx) <= tol).all()
        assert (gr.dweight is None) == (w is None) and (gr.dbias is None) == (not bias)
        if w is not None:
            assert gr.dweight.dtype == gdt
            assert (np.abs(host(gr.dweight) - dw) <= tw + HALF[gdt] * np.abs(dw)).all()
        if bias:
            assert (np.abs(host(gr.dbias) - db) <= tb + HALF[gdt] * np.abs(db)).all()
        again = g.layer_norm_backward(dy, x, stats, w, bias_grad=bias, grad_dtype=gdt)
        assert torch.equal(again.dx, gr.dx)
        assert w is None or torch.equal(again.dweight, gr.dweight)
        assert not bias or torch.equal(again.dbias, gr.dbias)


def test_layer_norm_backward_workspace_edges():
    """Nothing is read from the workspace that was not written, or written past its end."""
    import grouped_gemm_histogram_amd as g
    for T, H in ((1, 2880), (3, 64), (700, 130), (2000, 2881)):
        x, dy, w = rand(1, T, H), rand(2, T, H), rand(3, H)
        _, stats = g.layer_norm(x, w, return_stats=True)
        want = g.layer_norm_backward(dy, x, stats, w, bias_grad=True)
        need = g.layer_norm_backward_workspace_bytes(T, H)
        buf = torch.full((need // 4 + 64,), float("nan"), device=DEV)
        buf[need // 4:] = 7.0
        ws = buf[:need // 4].view(torch.uint8)
        got = g.layer_norm_backward(dy, x, stats, w, bias_grad=True, workspace=ws)
        for a, b in ((got.dx, want.dx), (got.dweight, want.dweight), (got.dbias, want.dbias)):
            assert torch.equal(a, b)
        assert (buf[need // 4:] == 7.0).all()
        # dx in place of dy, and of x
        for inp in (dy, x):
            d, v = dy.clone(), x.clone()
            buf2 = d if inp is dy else v
            g.layer_norm_backward(d, v, stats, w, bias_grad=True, dx=buf2)
            assert torch.equal(buf2, want.dx)
        with pytest.raises(RuntimeError, match="MOE_ERR_WORKSPACE"):
            g.layer_norm_backward(dy, x, stats, w, workspace=ws[:need - 4])


def rng_tensor(seed, offset=0):
    s = lambda v: v - (1 << 64) if v >= 1 << 63 else v
    return torch.tensor([s(seed), s(offset)], dtype=torch.int64, device=DEV)


def check_dropped(out, x, seed, offset, p, residual):
    """out against the oracle: dropped elements are the residual exactly, kept ones within rounding."""
    xs = host(x)
    ref = odrop.dropout_add(xs, seed, offset, p, host(residual))
    keep = odrop.keep_mask(x.numel(), seed, offset, p).reshape(xs.shape)
    got = host(out)
    r = torch.zeros_like(out) if residual is None else residual.to(out.dtype)
    assert torch.equal(out[torch.from_numpy(~keep).to(DEV)], r[torch.from_numpy(~keep).to(DEV)])
    scale = 0.0 if p >= 1.0 else 1.0 / (1.0 - p)
    # rounding of the scale to f32, of the sum to f32, and to out's type
    tol = U * np.abs(xs * scale) + (U + HALF[out.dtype]) * np.abs(ref)
    assert (np.abs(got - ref) <= tol)[keep].all()


@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 2048, 2049, 5003])
@pytest.mark.parametrize("xdt,rdt,odt", [
    (torch.bfloat16, None, torch.bfloat16), (torch.float32, None, torch.float32),
    (torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.float32),
    (torch.float32, torch.bfloat16, torch.float32), (torch.float32, torch.float32, torch.bfloat16),
    (torch.bfloat16, None, torch.float32), (torch.float32, None, torch.bfloat16)])
def test_dropout_add(n, xdt, rdt, odt):
    import grouped_gemm_histogram_amd as g
    for p, seed, offset in ((0.1, 3, 0), (0.5, (1 << 64) - 5, (1 << 32) - 3), (0.0, 1, 1), (1.0, 1, 1),
                            (1.0 / 65536, 11, (1 << 64) - 2)):
        say(f"dropout_add n={n} {xdt} {rdt} {odt} p={p}")
        x = rand(n, n, dtype=xdt)
        r = None if rdt is None else rand(n + 1, n, dtype=rdt)
        out = g.dropout_add(x, rng_tensor(seed, offset), p, residual=r, out_dtype=odt)
        assert out.dtype == odt
        check_dropped(out, x, seed, offset, p, r)
        # the gradient meets the same mask
        dx = g.dropout_add_backward(torch.ones(n, device=DEV), rng_tensor(seed, offset), p)
        assert torch.equal(dx != 0, torch.from_numpy(odrop.keep_mask(n, seed, offset, p)).to(DEV))


def test_dropout_threshold_ties():
    """Thresholds placed at the uniforms of single elements: the low halves decide."""
    import grouped_gemm_histogram_amd as g
    n, seed = 256, 77
    u = odrop.uniforms(n, seed, 5)
    x = torch.ones(n, device=DEV)
    for i in (0, 3, 100, 255):
        for d in (0, 1):   # p * 2^32 = u[i] + d is exact in a double
            p = (int(u[i]) + d) / 2.0 ** 32
            out = g.dropout_add(x, rng_tensor(seed, 5), p)
            assert torch.equal(out != 0, torch.from_numpy(u >= int(u[i]) + d).to(DEV))


def test_dropout_special_values_in_place_and_refusals():
    import grouped_gemm_histogram_amd as g
    n = 4096
    x = torch.full((n,), float("nan"), device=DEV)
    keep = torch.from_numpy(odrop.keep_mask(n, 9, 0, 0.5)).to(DEV)
    r = rand(1, n)
    out = g.dropout_add(x, rng_tensor(9), 0.5, residual=r)
    assert torch.isnan(out[keep]).all() and torch.equal(out[~keep], r[~keep])
    assert torch.equal(g.dropout_add(x, rng_tensor(9), 1.0, residual=r), r)
    x = rand(2, n)
    want = g.dropout_add(x, rng_tensor(9), 0.5, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(g.dropout_add(a, rng_tensor(9), 0.5, residual=r, out=a), want)
    assert torch.equal(g.dropout_add(x, rng_tensor(9), 0.5, residual=b, out=b), want)
    assert torch.equal(g.dropout_add(x, rng_tensor(9).view(torch.uint64), 0.5, residual=r), want)
    assert g.dropout_add(torch.empty(0, 5, device=DEV), rng_tensor(9), 0.5).shape == (0, 5)
    assert g.dropout_counters(0) == 0 and g.dropout_counters(8) == 1 and g.dropout_counters(9) == 2
    with pytest.raises(RuntimeError, match="MOE_ERR_INVALID_ARG"):
        g.dropout_add(x, rng_tensor(9), 1.5)
    with pytest.raises(ValueError, match="rng"):
        g.dropout_add(x, torch.zeros(2, device=DEV), 0.5)
    with pytest.raises(ValueError, match="residual"):
        g.dropout_add(x, rng_tensor(9), 0.5, residual=r[:5])
    with pytest.raises(RuntimeError, match="overlaps"):
        g.dropout_add(x[:2000], rng_tensor(9), 0.5, out=x[1024:3024])
    with pytest.raises(RuntimeError, match="aligned"):
        g.dropout_add(x[1:9], rng_tensor(9), 0.5)


@pytest.mark.parametrize("T,H,k,E", [(1, 8, 1, 8), (3, 520, 4, 8), (70, 136, 2, 32), (1100, 16, 8, 16)])
@pytest.mark.parametrize("ydt,rdt,odt", [
    (torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.float32),
    (torch.float32, torch.float32, torch.float32), (torch.float32, torch.bfloat16, torch.bfloat16),
    (torch.bfloat16, None, torch.bfloat16), (torch.float32, None, torch.bfloat16)])
def test_combine_dropout(T, H, k, E, ydt, rdt, odt):
    import grouped_gemm_histogram_amd as g
    say(f"unpermute_combine_dropout T={T} H={H} k={k} {ydt} {rdt} {odt}")
    logits = rand(T, T, E)
    V = T * k - T * k // 5                    # the last fifth of the rows are sentinels
    ids, w = g.route_topk(logits, k, V)
    offsets, _, row_pos = g.build_offsets(ids, E)
    y = rand(5, T * k, H, dtype=ydt)
    y[V:] = float("nan")                      # never read
    r = None if rdt is None else rand(6, T, H, dtype=rdt)
    seed, offset, p = 21, (1 << 32) - 2, 0.3
    out = g.unpermute_combine_dropout(y, row_pos, w, offsets, k, rng_tensor(seed, offset), p, residual=r,
                                      out_dtype=odt)
    # the f32 sums of the plain combine, which the fused form drops without rounding them
    sums = g.unpermute_combine(y, row_pos, w, offsets, k, out_dtype=torch.float32)
    check_dropped(out, sums, seed, offset, p, r)
    want = g.dropout_add(sums, rng_tensor(seed, offset), p, residual=r, out_dtype=odt)
    assert torch.equal(out, want)


def test_on_another_stream_and_two_at_once():
    """Each call runs on the current stream: two streams at once, each with its own inputs."""
    import grouped_gemm_histogram_amd as g
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [rand(i, 2000, 2880, dtype=torch.bfloat16) for i in range(2)]
    w = rand(9, 2880)
    want = []
    for x in xs:
        y, st = g.layer_norm(x, w, return_stats=True)
        want.append((y, g.layer_norm_backward(x, x, st, w), g.dropout_add(x, rng_tensor(4), 0.5)))
    torch.cuda.synchronize()
    got = [None, None]
    for rep in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                y, st = g.layer_norm(xs[i], w, return_stats=True)
                got[i] = (y, g.layer_norm_backward(xs[i], xs[i], st, w), g.dropout_add(xs[i], rng_tensor(4), 0.5))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1].dx, b[1].dx) and torch.equal(a[2], b[2])
            assert torch.equal(a[1].dweight, b[1].dweight)


def test_arrays_past_32_bits():
    """Element and byte offsets past 2^31 and 2^32: the last rows as in a call on them alone."""
    import grouped_gemm_histogram_amd as g
    T, H, n = 140000, 32768, 600                       # 4.59e9 elements, bf16
    say("layer_norm past 32 bits")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:n], x[-n:] = rand(1, n, H, dtype=torch.bfloat16), rand(2, n, H, dtype=torch.bfloat16)
    y, stats = g.layer_norm(x, return_stats=True)
    for rows in (slice(0, n), slice(T - n, T)):
        want, ws = g.layer_norm(x[rows], return_stats=True)
        assert torch.equal(y[rows], want) and torch.equal(stats.rstd[rows], ws.rstd)
    assert (y[n:-n:1000] == 0).all()
    say("layer_norm_backward past 32 bits")
    dx = g.layer_norm_backward(y, x, stats, dx=y).dx    # dy = y
    for rows in (slice(0, n), slice(T - n, T)):
        dy, s = g.layer_norm(x[rows], return_stats=True)
        assert torch.equal(dx[rows], g.layer_norm_backward(dy, x[rows], s).dx)
    del dx, y
    say("dropout_add past 32 bits")
    out = g.dropout_add(x, rng_tensor(3, 7), 0.4)
    start = (T - n) * H
    assert torch.equal(out[-n:], g.dropout_add(x[-n:], rng_tensor(3, 7 + start // 8), 0.4))
    assert torch.equal(out[:n], g.dropout_add(x[:n], rng_tensor(3, 7), 0.4))
    del out
    say("unpermute_combine_dropout past 32 bits")
    k = 2
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    w = torch.full((T // k, k), 0.5, device=DEV)
    off = torch.tensor([0, T, T], dtype=torch.int32, device=DEV)
    out = g.unpermute_combine_dropout(x, pos, w, off, k, rng_tensor(3, 7), 0.4)
    at = (T // k - n // k) * H
    want = g.unpermute_combine_dropout(x[-n:], pos[:n], w[:n // k], off.clamp(max=n), k, rng_tensor(3, 7 + at // 8), 0.4)
    assert torch.equal(out[-n // k:], want)
