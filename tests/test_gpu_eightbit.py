"""8-bit integers on the GPU: the coding, the grouped product and the layer against the oracle.

Tolerances (u = 2^-24).  Codes and scales are defined to the bit.  A product's sum is an exact integer; its
conversion and the two scales are off by u each, so an f32 result by 3 u of itself (3.1 with the
products of errors), a bf16 one by half a step, 2^-8, more.  SiLU * up: an error of 3.1 u of the gate g moves silu(g)
by at most (1 + |g|) of that share; exp(-g) is exp2 of a rounded product with a rounded constant, 1.5 u |g| of
itself; the exponential, sum, division and products add less than 8 u; up's 3.1 u.  Where exp(-g) leaves
f32's range (g < -88.7) the result is 0 instead of at most 2^-121 |up|.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, row_rel_err, say
from oracle import eightbit as o8

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def dev(a, dtype=None):
    t = torch.as_tensor(np.asarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def codes(rng, *shape):
    return rng.integers(-128, 128, shape, dtype=np.int64).astype(np.int8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,H", [(1, 16), (3, 2880), (5, 32768), (600, 7168), (513, 48), (700, 272), (512, 24592)])
def test_quantize_rows(rows, H, dtype):
    say("quantize", rows, H, dtype)
    rng = np.random.default_rng(rows * H)
    x = torch.from_numpy((rng.normal(size=(rows, H)) * np.exp(rng.normal(size=(rows, 1)))).astype(np.float32)).to(dtype)
    x[0, H // 2] = 2 * x[0].abs().max()                          # its half is next to a tie
    x[0, 1] = x[0, H // 2] / 2
    if rows > 2:
        x[1] = 0
        x[2] = x[2] * 2.0 ** -110                                # below the least scale: zeros
    q, s = g.quantize_rows_eightbit(x.to(DEV))
    rq, rs = o8.quantize_rows(x.float().numpy())
    assert (s.cpu().numpy() == rs).all()
    assert (q.cpu().numpy() == rq).all()


def test_quantize_rows_weights_and_bad_rows():
    w = torch.randn(3, 40, 64, device=DEV)
    w[1, 5, 7] = float("nan")
    w[2, 0, 63] = float("-inf")
    q, s = g.quantize_rows_eightbit(w)
    assert q.shape == w.shape and s.shape == (3, 40)
    s = s.cpu()
    assert torch.isnan(s[1, 5]) and torch.isinf(s[2, 0]) and int((~torch.isfinite(s)).sum()) == 2
    ok = torch.isfinite(s)
    rq, rs = o8.quantize_rows(w.cpu()[ok].numpy())
    assert (q.cpu()[ok].numpy() == rq).all() and (s[ok].numpy() == rs).all()
    e = torch.empty(0, 32, device=DEV)
    q, s = g.quantize_rows_eightbit(e)
    assert q.shape == (0, 32) and s.shape == (0,)


# rows of each expert, tail (rows without an expert), N, K: few rows, some, many; K of one MFMA's share and less,
# columns that end inside a tile
SHAPES = [
    ([1], 0, 16, 16),
    ([0, 3, 0, 1], 2, 48, 48),
    ([2, 0, 5, 8, 1, 0], 3, 96, 2880),
    ([20, 0, 33, 7], 5, 64, 208),
    ([31, 30, 32], 0, 200, 128),
    ([300, 0, 190, 1], 9, 208, 144),
    ([193, 400], 0, 400, 2064),
    ([700], 1, 592, 80),
    ([0, 0], 4, 32, 32),
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,tail,N,K", SHAPES)
def test_grouped_gemm(counts, tail, N, K, out, silu, gather):
    say("gemm", counts, tail, N, K, out, silu, gather)
    rng = np.random.default_rng(sum(counts) * K + N)
    E, V = len(counts), sum(counts)
    M = V + tail
    off = np.concatenate([[0], np.cumsum(counts)])
    A_rows = max(1, M // 2) if gather else M + 1
    a, b = codes(rng, A_rows, K), codes(rng, E, N, K)
    sa = (0.02 * (rng.random(A_rows) + 0.1)).astype(np.float32)
    sb = (0.02 * (rng.random((E, N)) + 0.1)).astype(np.float32)
    rows = rng.integers(0, A_rows * 3, M) if gather else None
    src = rows // 3 if gather else np.arange(M)
    n_out = N // 2 if silu else N
    call = lambda: g.grouped_gemm_eightbit(
        dev(a), dev(sa), dev(b), dev(sb), dev(off, torch.int32), "silu_mul" if silu else "none", out_dtype=out,
        **(dict(gather_rows=dev(rows, torch.int32), gather_div=3) if gather else
           dict(out=torch.full((A_rows, n_out), 7.0, dtype=out, device=DEV))))
    if n_out * out.itemsize % 16:   # rows of C are whole 16 bytes: refused
        with pytest.raises(RuntimeError, match="16 bytes"):
            call()
        return
    got = call().double().cpu().numpy()
    assert got.shape == ((M if gather else A_rows), n_out)
    assert (got[V:] == 0).all()
    ref = o8.grouped_gemm(a[src], sa[src], b, sb, off, M, silu)
    half = 2.0 ** -8 if out == torch.bfloat16 else 0.0
    if silu:
        ref, gate, up = ref
        tol = np.abs(ref) * (3.1 * U * (2 + np.abs(gate)) + (8 + 1.5 * np.abs(gate)) * U + half) + 2.0 ** -121 * np.abs(up)
    else:
        tol = np.abs(ref) * (3.1 * U + half)
    bad = np.abs(got[:M] - ref) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got[:M] - ref)[bad].max()))


@pytest.mark.parametrize("K", [131056, 4096])
def test_sums_at_the_ends_of_32_bits(K):
    """Every product 2^14 or -127 * 128: sums next to 2^31, exact."""
    a = np.full((4, K), -128, np.int8)
    b = np.full((1, 16, K), -128, np.int8)
    b[0, 1] = 127
    b[0, 2, 1::2] = 127
    one = np.ones(4, np.float32)
    got = g.grouped_gemm_eightbit(dev(a), dev(one), dev(b), dev(np.ones((1, 16), np.float32)),
                                  dev([0, 4], torch.int32), out_dtype=torch.float32).cpu().numpy()
    ref = (a.astype(np.int64) @ b[0].astype(np.int64).T).astype(np.float32)   # integers of 31 bits, rounded once
    assert (got == ref).all()


def test_bad_maps_and_offsets_stay_inside():
    rng = np.random.default_rng(5)
    a, b = codes(rng, 6, 32), codes(rng, 2, 32, 32)
    sa, sb = np.ones(6, np.float32), np.ones((2, 32), np.float32)
    rows = np.array([-5, 100, 3, 2 ** 31 - 1], np.int64)
    got = g.grouped_gemm_eightbit(dev(a), dev(sa), dev(b), dev(sb), dev([0, 2, 4], torch.int32),
                                  gather_rows=dev(rows, torch.int32), out_dtype=torch.float32).cpu().numpy()
    src = np.clip(rows, 0, 5)
    assert (got == o8.grouped_gemm(a[src], sa[src], b, sb, [0, 2, 4], 4, False)).all()
    got = g.grouped_gemm_eightbit(dev(a), dev(sa), dev(b), dev(sb), dev([-3, 4, 99], torch.int32), out_dtype=torch.float32)
    assert (got.cpu().numpy() == o8.grouped_gemm(a, sa, b, sb, [0, 4, 6], 6, False)).all()


@pytest.mark.parametrize("T,H,I,E,k,valid,out", [
    (1, 32, 16, 4, 2, -1, torch.bfloat16),
    (7, 208, 272, 16, 4, 17, torch.float32),
    (64, 256, 192, 8, 2, -1, torch.bfloat16),
    (300, 512, 256, 4, 2, 401, torch.float32),
    (33, 64, 48, 1, 1, -1, torch.float32),
    (5, 64, 48, 8, 3, 0, torch.bfloat16),
])
def test_layer(T, H, I, E, k, valid, out):
    """A hidden value next to a border of bf16 (one in some thousands) may round the other way, and its code
    then be one off: 1/127 of the row's largest h in a sum of I products, which is well below the bf16 layer's
    1e-2 of the output row's largest value."""
    say("layer", T, H, I, E, k, valid)
    rng = np.random.default_rng(T * H)
    x = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    w13, s13 = o8.quantize_rows((rng.normal(size=(E, 2 * I, H)) / H ** 0.5).astype(np.float32))
    w2, s2 = o8.quantize_rows((rng.normal(size=(E, H, I)) / I ** 0.5).astype(np.float32))
    args = (x.to(DEV), dev(logits), dev(w13), dev(s13), dev(w2), dev(s2), k)
    got, aux = g.forward_eightbit(*args, num_valid_rows=valid, out_dtype=out, return_aux=True)
    ref = o8.forward(x.float().numpy(), logits, w13, s13, w2, s2, k, valid)
    assert int(aux.offsets[-1]) == (T * k if valid < 0 else valid)
    err = row_rel_err(np32(got), ref)
    say("  error", err)
    assert err < 1e-2
    assert (np32(got)[np.abs(ref).max(axis=1) == 0] == 0).all()
    again = g.forward_eightbit(*args, num_valid_rows=valid, out_dtype=out)
    assert torch.equal(got, again)


def test_layer_is_its_steps():
    """The layer's output equals the entry points called one by one, to the bit."""
    rng = np.random.default_rng(11)
    T, H, I, E, k = 40, 256, 128, 8, 2
    x = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(DEV)
    w13, s13 = g.quantize_rows_eightbit(torch.from_numpy(rng.normal(size=(E, 2 * I, H)).astype(np.float32)).to(DEV) * 0.05)
    w2, s2 = g.quantize_rows_eightbit(torch.from_numpy(rng.normal(size=(E, H, I)).astype(np.float32)).to(DEV) * 0.05)
    out = g.forward_eightbit(x, logits, w13, s13, w2, s2, k)
    ids, w = g.route_topk(logits, k)
    off, order, pos = g.build_offsets(ids, E)
    xq, xs = g.quantize_rows_eightbit(x)
    h = g.grouped_gemm_eightbit(xq, xs, w13, s13, off, "silu_mul", gather_rows=order, gather_div=k)
    hq, hs = g.quantize_rows_eightbit(h)
    y = g.grouped_gemm_eightbit(hq, hs, w2, s2, off)
    assert torch.equal(out, g.unpermute_combine(y, pos, w, off, k))


def test_replayed_graph_and_other_stream():
    rng = np.random.default_rng(12)
    T, H, I, E, k = 20, 128, 64, 8, 2
    x = torch.from_numpy(rng.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
    logits = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32)).to(DEV)
    w13, s13 = g.quantize_rows_eightbit(torch.randn(E, 2 * I, H, device=DEV))
    w2, s2 = g.quantize_rows_eightbit(torch.randn(E, H, I, device=DEV))
    ws = torch.empty(g.forward_eightbit_workspace_bytes(T, H, I, E, k), dtype=torch.uint8, device=DEV)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    call = lambda: g.forward_eightbit(x, logits, w13, s13, w2, s2, k, out=out, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        out.zero_()
        x.copy_(torch.randn(T, H, device=DEV)) if i else None
        graph.replay()
        torch.cuda.synchronize()
        want = g.forward_eightbit(x, logits, w13, s13, w2, s2, k)
        assert torch.equal(out, want)
        if i == 0:
            assert torch.equal(out, first)


def test_refusals():
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)
    f = lambda *s: torch.ones(*s, device=DEV)
    off = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        g.grouped_gemm_eightbit(i8(2, 32).float(), f(2), i8(1, 16, 32), f(1, 16), off)
    with pytest.raises(ValueError):
        g.grouped_gemm_eightbit(i8(2, 32), f(3), i8(1, 16, 32), f(1, 16), off)
    with pytest.raises(ValueError):
        g.grouped_gemm_eightbit(i8(2, 32), f(2), i8(1, 16, 48), f(1, 16), off)
    with pytest.raises(ValueError):
        g.grouped_gemm_eightbit(i8(2, 32), f(2), i8(1, 16, 32), f(1, 15), off)
    with pytest.raises(ValueError):
        g.grouped_gemm_eightbit(i8(4, 32)[::2], f(2), i8(1, 16, 32), f(1, 16), off)
    with pytest.raises(RuntimeError):
        g.grouped_gemm_eightbit(i8(2, 24), f(2), i8(1, 16, 24), f(1, 16), off)
    with pytest.raises(RuntimeError):
        g.quantize_rows_eightbit(f(2, 24))
    with pytest.raises(ValueError):
        g.forward_eightbit(f(2, 32), f(2, 1), i8(1, 32, 32), f(1, 32), i8(1, 32, 16), f(1, 32), 1)
