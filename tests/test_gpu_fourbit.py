"""4-bit expert products on the GPU against the float64 oracle: coding, grouped products, the layer.

Tolerances of random inputs (u = 2^-24).  mxfp4 operands are exact bf16 values, so a product
is off by the roundings of a sum of K terms, at most 2 K u times sum |a w| (2 u per addition also
covers an accumulator that truncates).  int4 sums a * (128 + code) and a * 136 over 32 channels,
each term at most 143 |a|, then scales: at most 2 (2 * 32 + 2) u * 143 * scale * sum |a| per group,
and the sum over groups.  SiLU * up passes an error of the gate on by at most 1.1 |up| and one of
up by |silu(gate)|.  Its own rounding: exp(-g) is exp2(-g log2 e), whose argument is rounded (u
of it) with a rounded constant (u / 2), so exp is off by 1.5 u ln 2 log2 e |g| = 1.5 u |g| of itself;
the exponential, sum, division and product add less than 8 u.  Where exp(-g) leaves f32's range
(g < -88.7) the result is 0 instead of at most 88.8 * 2^-128 |up| < 2^-121 |up|.
"""
import numpy as np
import pytest
import torch

from helpers import TOL, row_rel_err, say
from oracle import dropout as odrop, fourbit as ofb, layer as olayer, norm as onorm
from oracle.layer import ExpertWeights
from workloads import generate, get_config, small_variant

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FORMATS = [("mxfp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)]


def SILU(g):
    return 8 * U + 1.5 * U * np.abs(g)


def host(t):
    return t.detach().to("cpu", torch.float64).numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def weights(E, N, K, fmt, group, seed, exact=False):
    """Codes of every value; exact: scales are powers of two near 1."""
    g = gen(seed)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    if fmt == "mxfp4":
        scales = torch.randint(126, 129, (E, N, K // 32), generator=g).to(torch.uint8)
        if not exact:
            scales = torch.randint(110, 125, (E, N, K // 32), generator=g).to(torch.uint8)
    else:
        scales = 2.0 ** torch.randint(-1, 2, (E, N, K // group), generator=g).float()
        if not exact:
            scales = 0.01 * (0.5 + torch.rand(E, N, K // group, generator=g))
    return codes, scales


def offsets_of(counts, tail):
    off = np.zeros(len(counts) + 1, np.int64)
    off[1:] = np.cumsum(counts)
    return off, int(off[-1]) + tail


def reference(a, codes, scales, off, silu, exact=False):
    """(result, tolerance of an f32 result) [M, N_out] for permuted rows a [M, K]; exact: the
    products' sums are."""
    M, E = a.shape[0], len(off) - 1
    N = codes.shape[1]
    n_out = N // 2 if silu else N
    ref, tol = np.zeros((M, n_out)), np.zeros((M, n_out))
    K = a.shape[1]
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        w = ofb.dequantize(codes[e].numpy(), scales[e].numpy())
        acc = a[lo:hi] @ w.T
        if scales.dtype == torch.uint8:
            err = 2 * K * U * (np.abs(a[lo:hi]) @ np.abs(w).T)
        else:
            G = scales.shape[2]
            s = np.abs(scales[e].double().numpy())
            asum = np.abs(a[lo:hi]).reshape(hi - lo, G, -1).sum(2)
            err = 2 * (66 + K // 32) * U * 143 * (asum @ s.T)
        if exact:
            err = np.zeros_like(acc)
        if silu:
            g, u = acc[:, :n_out], acc[:, n_out:]
            sg = g / (1 + np.exp(-g))
            tol[lo:hi] = 1.1 * np.abs(u) * err[:, :n_out] + np.abs(sg) * err[:, n_out:] + SILU(g) * np.abs(sg * u)
            tol[lo:hi] += 2.0 ** -121 * np.abs(u)
            tol[lo:hi] += 1.1 * err[:, :n_out] * err[:, n_out:]
            acc = sg * u
        else:
            tol[lo:hi] = err
        ref[lo:hi] = acc
    return ref, tol


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize(fmt, group, dtype):
    import grouped_gemm_histogram_amd as g
    say(f"quantize_fourbit {fmt} {group} {dtype}")
    w = (torch.randn(3, 5, 256, generator=gen(1)) * 0.05).to(dtype)
    w[0, 0] = 0.0
    w[1, 2, :group] *= 1e-30
    w[2, 1] = torch.arange(256).float().to(dtype) / 8 - 16      # ties
    w[2, 2, :32] = torch.tensor([0.25, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0, 6.0, 7.9, -0.0] + [0.0] * 20)
    codes, scales = g.quantize_fourbit(w.to(DEV), fmt, group)
    rc, rs = ofb.quantize(w.float().numpy(), fmt, group)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)


# rows per expert (and rows without an expert): none, single rows, both sides of 16 and of 64
COUNTS = [([1], 0), ([0, 3, 0, 1], 2), ([16, 17, 0, 15], 1), ([0, 0, 5], 0), ([0, 0], 7), ([64, 65, 1, 130], 33),
          ([1] * 70 + [0] * 30, 3)]


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts,tail", COUNTS)
def test_matvec_exact(fmt, group, silu, counts, tail):
    """Small whole activations and power-of-two scales: every f32 sum is exact, whatever its order."""
    import grouped_gemm_histogram_amd as g
    for N, K in ((2, 128), (34, 384), (80, 128 * 7)):
        K = K if group > 32 else K - 32 if K > 128 else K      # a last step of one to four groups
        E = len(counts)
        off, M = offsets_of(counts, tail)
        say(f"matvec exact {fmt} {group} silu={silu} counts={counts[:6]} N={N} K={K}")
        codes, scales = weights(E, N, K, fmt, group, N + K, exact=True)
        a = torch.randint(-2, 3, (M, K), generator=gen(5)).to(torch.bfloat16)
        ref, tol = reference(host(a), codes, scales, off, silu, exact=True)
        out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV),
                                       torch.from_numpy(off).to(torch.int32).to(DEV), "silu_mul" if silu else "none",
                                       out_dtype=torch.float32)
        got = host(out)
        if silu:   # the epilogue rounds; the products are exact
            assert (np.abs(got - ref) <= tol).all()
        else:
            np.testing.assert_array_equal(got, ref)
        assert (got[off[-1]:] == 0).all()


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("N,K", [(30, 2880), (5760, 256), (18, 4096), (256, 7168)])
def test_matvec_random(fmt, group, silu, N, K):
    import grouped_gemm_histogram_amd as g
    if K % group:
        K = K // group * group
    counts, tail = [3, 0, 1, 20, 9], 2
    off, M = offsets_of(counts, tail)
    say(f"matvec {fmt} {group} silu={silu} N={N} K={K}")
    codes, scales = weights(5, N, K, fmt, group, N, exact=False)
    k = 3
    tokens = torch.randn(M, K, generator=gen(2)).to(torch.bfloat16)
    rows = torch.randperm(M * k, generator=gen(3))[:M].to(torch.int32)
    dev = [t.to(DEV) for t in (tokens, codes, scales, rows, torch.from_numpy(off).to(torch.int32))]
    epi = "silu_mul" if silu else "none"
    ref, tol = reference(host(tokens)[rows.numpy() // k], codes, scales, off, silu)
    out = g.grouped_matvec_fourbit(dev[0], dev[1], dev[2], dev[4], epi, gather_rows=dev[3], gather_div=k,
                                   out_dtype=torch.float32)
    assert (np.abs(host(out) - ref) <= tol + U * np.abs(ref)).all()
    b16 = g.grouped_matvec_fourbit(dev[0], dev[1], dev[2], dev[4], epi, gather_rows=dev[3], gather_div=k)
    assert torch.equal(b16, out.to(torch.bfloat16))
    # rows given in permuted order, into a buffer of NaN: the same bits, and zeros past the last valid row
    permuted = dev[0][(dev[3] // k).long()].contiguous()
    buf = torch.full_like(b16, float("nan"))
    g.grouped_matvec_fourbit(permuted, dev[1], dev[2], dev[4], epi, out=buf)
    assert torch.equal(buf, b16) and (buf[off[-1]:] == 0).all()


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("counts", [[2, 0, 1], [9, 12, 5], [30, 41, 17]])
@pytest.mark.parametrize("silu", [False, True])
def test_matvec_long_rows_exact(fmt, group, counts, silu):
    """Channels past what the streaming kernel holds (7168), and that many exactly, at few, some and many
    rows per expert."""
    import grouped_gemm_histogram_amd as g
    off, M = offsets_of(counts, 1)
    for K in (7168, 7296, 14336):
        say(f"matvec long {fmt} {group} counts={counts} silu={silu} K={K}")
        codes, scales = weights(3, 34, K, fmt, group, K, exact=True)
        a = torch.randint(-2, 3, (M, K), generator=gen(6)).to(torch.bfloat16)
        ref, tol = reference(host(a), codes, scales, off, silu, exact=True)
        out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV),
                                       torch.from_numpy(off).to(torch.int32).to(DEV), "silu_mul" if silu else "none",
                                       out_dtype=torch.float32)
        assert (np.abs(host(out) - ref) <= tol).all()


def test_matvec_longest_rows_and_beyond():
    import grouped_gemm_histogram_amd as g
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for fmt, group, K in (("int4", 32, 16128), ("int4", 64, 32512), ("int4", 128, 65280), ("mxfp4", 32, 65280)):
        codes, scales = weights(1, 4, K, fmt, group, K, exact=True)
        a = (torch.arange(K) % 97 == 0).to(torch.bfloat16)[None]      # few ones: sums stay exact
        ref, tol = reference(host(a), codes, scales, np.array([0, 1]), True, exact=True)
        out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV), off, "silu_mul",
                                       out_dtype=torch.float32)
        assert (np.abs(host(out) - ref) <= tol).all(), fmt
        long = torch.zeros(1, 2 * K + 512, dtype=torch.bfloat16, device=DEV)
        codes, scales = (t.to(DEV) for t in weights(1, 4, 2 * K + 512, fmt, group, 1))
        with pytest.raises(RuntimeError, match="MOE_ERR_UNSUPPORTED"):
            g.grouped_matvec_fourbit(long, codes, scales, off, "silu_mul")


def test_matvec_same_row_many_times_and_bad_maps():
    """A row map may repeat rows; entries outside A are clamped into it."""
    import grouped_gemm_histogram_amd as g
    codes, scales = weights(2, 32, 64, "int4", 32, 1, exact=True)
    a = torch.randint(-2, 3, (4, 64), generator=gen(1)).to(torch.bfloat16)
    rows = torch.tensor([2, 2, 2, 7, 1000000, -5], dtype=torch.int32)
    off = np.array([0, 4, 6])
    want, _ = reference(host(a)[[2, 2, 2, 3, 3, 0]], codes, scales, off, False)
    out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV),
                                   torch.from_numpy(off).to(torch.int32).to(DEV), gather_rows=rows.to(DEV),
                                   out_dtype=torch.float32)
    np.testing.assert_array_equal(host(out), want)


@pytest.mark.parametrize("fmt,group", [("mxfp4", 32), ("int4", 128)])
def test_matvec_arrays_past_32_bits(fmt, group):
    """The last expert of weights past 4 GiB, and the last rows of an output past 4 GiB."""
    import grouped_gemm_histogram_amd as g
    E, N, K = 72, 65536, 2048                          # 64 MiB of codes an expert
    say(f"matvec past 32 bits: weights {fmt}")
    gd = torch.Generator(device=DEV).manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gd, device=DEV, dtype=torch.uint8)
    if fmt == "mxfp4":
        scales = torch.randint(120, 125, (E, N, K // 32), generator=gd, device=DEV, dtype=torch.uint8)
    else:
        scales = torch.rand(E, N, K // group, generator=gd, device=DEV)
    a = torch.randn(9, K, generator=gen(2)).to(torch.bfloat16).to(DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 9
    one = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    for epi in ("none", "silu_mul"):
        out = g.grouped_matvec_fourbit(a, codes, scales, off, epi, out_dtype=torch.float32)
        want = g.grouped_matvec_fourbit(a, codes[-1:].clone(), scales[-1:].clone(), one, epi, out_dtype=torch.float32)
        assert torch.equal(out, want) and out.abs().sum() > 0
    say("matvec past 32 bits: output")
    M = 40000                                          # x 65536 bf16 columns
    codes, scales = codes[:1, :, :64].contiguous(), scales[:1, :, :128 // group].contiguous()
    a = torch.randn(M, 128, generator=gen(3)).to(torch.bfloat16).to(DEV)
    off = torch.tensor([0, M - 8], dtype=torch.int32, device=DEV)
    out = g.grouped_matvec_fourbit(a, codes, scales, off)
    for lo in (0, M - 40):                             # whole blocks of 16 rows, then a part of one
        hi = min(lo + 48, M - 8)
        want = g.grouped_matvec_fourbit(a[lo:hi], codes, scales, torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV))
        assert torch.equal(out[lo:hi], want)
    assert (out[M - 8:] == 0).all()


def test_offsets_that_do_not_ascend():
    """Such offsets are a mistake: no expert has rows then, and nothing past the output is written."""
    import grouped_gemm_histogram_amd as g
    codes, scales = weights(3, 32, 64, "int4", 32, 1, exact=True)
    a = torch.randint(-2, 3, (48, 64), generator=gen(2)).to(torch.bfloat16)
    buf = torch.full((48 + 64, 32), 7.0, device=DEV)
    say("offsets 0 40 8 44")
    out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV),
                                   torch.tensor([0, 40, 8, 44], dtype=torch.int32, device=DEV), out=buf[32:80])
    assert (out[44:] == 0).all()
    assert (buf[:32] == 7).all() and (buf[80:] == 7).all()


def test_mxfp4_smallest_scales():
    """Scale bytes 0 and 1, on codes whose values 2^-126 and up are normal bf16 numbers."""
    import grouped_gemm_histogram_amd as g
    row = torch.tensor([4 | 5 << 4, 6 | 7 << 4, 12 | 13 << 4, 14 | 15 << 4], dtype=torch.uint8).repeat(4)   # 2 3 4 6 and negatives
    c = row.view(1, 1, 16).repeat(1, 2, 1)
    s = torch.tensor([0, 1], dtype=torch.uint8).view(1, 2, 1)
    a = torch.zeros(8, 32)
    a[torch.arange(8), torch.arange(8)] = 2.0 ** 100
    out = g.grouped_matvec_fourbit(a.to(torch.bfloat16).to(DEV), c.to(DEV), s.to(DEV),
                                   torch.tensor([0, 8], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    want = ofb.dequantize(c[0].numpy(), s[0].numpy())[:, :8].T * 2.0 ** 100
    np.testing.assert_array_equal(host(out), want)


def test_mxfp4_scale_range():
    """Every scale byte at which all values are normal bf16 numbers, and the byte that means NaN."""
    import grouped_gemm_histogram_amd as g
    codes = torch.arange(16, dtype=torch.uint8)
    row = (codes[0::2] | (codes[1::2] << 4)).repeat(2)             # the sixteen codes twice: one group
    sb = [2, 64, 126, 127, 128, 200, 251, 255]                     # 6 * 2^124 is the largest value below 2^127
    N = len(sb)
    c = row.repeat(1, N, 1).view(1, N, 16)
    s = torch.tensor(sb, dtype=torch.uint8).view(1, N, 1)
    a = torch.zeros(16, 32)
    a[torch.arange(16), torch.arange(16)] = 1.0                    # row i picks channel i
    out = g.grouped_matvec_fourbit(a.to(torch.bfloat16).to(DEV), c.to(DEV), s.to(DEV),
                                   torch.tensor([0, 16], dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    want = ofb.dequantize(c[0].numpy(), s[0].numpy())[:, :16].T
    got = host(out)
    np.testing.assert_array_equal(got[:, :-1], want[:, :-1])
    assert np.isnan(got[:, -1]).all()


def test_refusals():
    import grouped_gemm_histogram_amd as g
    codes, scales = (t.to(DEV) for t in weights(2, 32, 64, "int4", 32, 1))
    a = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="K mismatch"):
        g.grouped_matvec_fourbit(a[:, :32].contiguous(), codes, scales, off)
    with pytest.raises(ValueError, match="scales"):
        g.grouped_matvec_fourbit(a, codes, scales[:, :16].contiguous(), off)
    with pytest.raises(ValueError, match="dtype"):
        g.grouped_matvec_fourbit(a.float(), codes, scales, off)
    with pytest.raises(ValueError, match="offsets"):
        g.grouped_matvec_fourbit(a, codes, scales, off[:2])
    with pytest.raises(RuntimeError, match="MOE_ERR_INVALID_ARG"):    # groups of 16
        g.grouped_matvec_fourbit(a, codes, scales.repeat(1, 1, 2).contiguous(), off)
    with pytest.raises(ValueError, match="group"):
        g.quantize_fourbit(torch.zeros(1, 4, 96, device=DEV), "int4", 64)
    with pytest.raises(ValueError, match="format"):
        g.quantize_fourbit(torch.zeros(1, 4, 96, device=DEV), "int8")
    assert g.grouped_matvec_fourbit(a[:0], codes, scales, torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (0, 32)


LAYERS = [("gptoss20b_bf16", 1, {}, "mxfp4", 32), ("gptoss20b_bf16", 8, dict(H=416, I=288), "int4", 32),
          ("gptoss20b_bf16", 70, dict(H=256, I=384), "int4", 128), ("sweep_bf16_v8192", 24, dict(I=256), "int4", 64),
          ("mixtral8x7b_bf16", 200, dict(H=512, I=320), "mxfp4", 32), ("gptoss20b_bf16", 0, dict(H=64, I=64), "mxfp4", 32)]


@pytest.mark.parametrize("name,T,kw,fmt,group", LAYERS)
def test_forward_fourbit(name, T, kw, fmt, group):
    """The layer on 4-bit weights against the oracle's layer on the values they stand for."""
    import grouped_gemm_histogram_amd as g
    cfg = small_variant(get_config(name), T).replace(**kw)
    say(f"forward_fourbit {cfg.name} T={T} H={cfg.H} I={cfg.I} {fmt} {group}")
    inp = generate(cfg, "cpu")
    dev = inp.to(DEV)
    q13, s13 = g.quantize_fourbit(dev.w13, fmt, group)
    q2, s2 = g.quantize_fourbit(dev.w2, fmt, group)
    out, aux = g.forward_fourbit(dev.x, dev.logits, q13, s13, q2, s2, cfg.k, cfg.num_valid_rows, cfg.renormalize,
                                 return_aux=True)
    assert out.shape == (T, cfg.H)
    if T == 0:
        assert int(aux.offsets.abs().sum()) == 0
        return
    W = ExpertWeights(ofb.dequantize(q13.cpu().numpy(), s13.cpu().numpy()),
                      ofb.dequantize(q2.cpu().numpy(), s2.cpu().numpy()))
    ref = olayer.forward(inp.x.float().numpy(), inp.logits.numpy(), W, cfg.k, cfg.num_valid_rows)
    np.testing.assert_array_equal(aux.topk_ids.cpu().numpy(), ref["ids"])
    np.testing.assert_array_equal(aux.offsets.cpu().numpy(), ref["offsets"])
    assert row_rel_err(host(out), ref["out"]) <= TOL["bf16"]
    f32 = g.forward_fourbit(dev.x, dev.logits, q13, s13, q2, s2, cfg.k, cfg.num_valid_rows, cfg.renormalize,
                            out_dtype=torch.float32)
    assert torch.equal(f32.to(torch.bfloat16), out)


def test_block_graph_replay():
    """norm -> router -> 4-bit layer -> dropout + residual captured and replayed: each replay equals the
    eager run on the same inputs and generator state, and a changed state gives a changed mask."""
    import grouped_gemm_histogram_amd as g
    T, H, I, E, k = 5, 512, 256, 16, 4
    cfg = small_variant(get_config("gptoss20b_bf16"), T).replace(H=H, I=I, E=E)
    inp = generate(cfg, DEV)
    q13, s13 = g.quantize_fourbit(inp.w13, "mxfp4")
    q2, s2 = g.quantize_fourbit(inp.w2, "mxfp4")
    x = inp.x.clone()
    w = torch.ones(H, device=DEV)
    wr = (torch.randn(E, H, generator=gen(1)) * 0.1).to(DEV)
    rng = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    out = torch.empty(T, H, device=DEV, dtype=torch.bfloat16)

    def block(xx, o):
        y = g.layer_norm(xx, w, rms=True)
        moe = g.forward_fourbit(y, torch.mm(y.float(), wr.t()).contiguous(), q13, s13, q2, s2, k)
        return g.dropout_add(moe, rng, 0.2, residual=xx, out=o)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, out)
    seen = []
    for i in range(4):
        rng[1] = i // 2 * g.dropout_counters(T * H)
        x.copy_(inp.x * (1 + i))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = block(x, torch.empty_like(out))
        assert torch.equal(out, want), f"replay {i}"
        seen.append(out == x)
    assert not torch.equal(seen[0], seen[2])


def test_backward_graph_replay():
    """The gradients captured and replayed, twice with new gradients, against eager calls."""
    import grouped_gemm_histogram_amd as g
    T, H = 600, 1000
    x = torch.randn(T, H, generator=gen(1)).to(torch.bfloat16).to(DEV)
    w = torch.randn(H, generator=gen(2)).to(DEV)
    dy = torch.randn(T, H, generator=gen(3)).to(torch.bfloat16).to(DEV)
    rng = torch.tensor([5, 0], dtype=torch.int64, device=DEV)
    _, stats = g.layer_norm(x, w, return_stats=True)
    step = lambda: g.layer_norm_backward(g.dropout_add_backward(dy, rng, 0.3), x, stats, w, bias_grad=True)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        dy.mul_(1.0 + i)
        rng[1] += 100
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)
        assert torch.equal(got.dbias, want.dbias)


def test_block_training_gradients():
    """norm -> router -> bf16 layer -> combine with dropout and residual, and its gradients, as a
    training step makes them, against the oracle's functions put together the same way (with
    the layer's own bf16 tolerances)."""
    import grouped_gemm_histogram_amd as g
    from oracle import backward as obwd
    T, H, I, E, k, p = 48, 256, 192, 8, 2, 0.25
    cfg = small_variant(get_config("gptoss20b_bf16"), T).replace(H=H, I=I, E=E, k=k)
    inp = generate(cfg, "cpu")
    dev = inp.to(DEV)
    w = 1.0 + 0.1 * torch.randn(H, generator=gen(1))
    b = 0.1 * torch.randn(H, generator=gen(2))
    wd, bd = w.to(DEV), b.to(DEV)
    rng = torch.tensor([17, 3], dtype=torch.int64, device=DEV)
    y, stats = g.layer_norm(dev.x, wd, bd, return_stats=True)
    ids, tw = g.route_topk(dev.logits, k)
    offsets, sorted_rows, row_pos = g.build_offsets(ids, E)
    h = g.grouped_gemm_gather(y, dev.w13, offsets, sorted_rows, k, "silu_mul")
    rows = g.grouped_gemm(h, dev.w2, offsets)
    out = g.unpermute_combine_dropout(rows, row_pos, tw, offsets, k, rng, p, residual=dev.x)
    dout = torch.randn(T, H, generator=gen(4)).to(torch.bfloat16)
    dmoe = g.dropout_add_backward(dout.to(DEV), rng, p)
    gr = g.backward(y, dev.w13, dev.w2, dmoe, tw, offsets, sorted_rows, row_pos, grad_dtype=torch.bfloat16)
    gn = g.layer_norm_backward(gr.dx, dev.x, stats, wd, bias_grad=True)
    torch.cuda.synchronize()

    f = lambda t: t.float().numpy()
    W = ExpertWeights(f(inp.w13), f(inp.w2))
    ry, rm, rr = onorm.layer_norm(f(inp.x), f(w), f(b))
    ref = olayer.forward(f(y.cpu()), inp.logits.numpy(), W, k)
    assert row_rel_err(host(y), ry) <= 2.0 ** -7
    want = odrop.dropout_add(ref["out"], 17, 3, p, host(inp.x))
    assert row_rel_err(host(out), want) <= TOL["bf16"]
    rdmoe = odrop.dropout_add(host(dout), 17, 3, p)
    assert row_rel_err(host(dmoe), rdmoe) <= 2.0 ** -8
    gref = obwd.backward(f(y.cpu()), ref["ids"], ref["w"], W, f(dmoe.cpu()))
    assert row_rel_err(host(gr.dx), gref["dx"]) <= 2e-2
    rdx, rdw, rdb = onorm.layer_norm_backward(gref["dx"], f(inp.x), rm, rr, f(w))
    # the layer's dx is within 2e-2 of its rows' largest entry: so are the norm's gradients of it,
    # whose linear map has row norms of at most rstd * max|w| (dx) and sums T independent rows (dweight)
    assert row_rel_err(host(gn.dx), rdx) <= 4e-2
    assert row_rel_err(host(gn.dweight)[None], rdw[None]) <= 4e-2
    assert row_rel_err(host(gn.dbias)[None], rdb[None]) <= 4e-2
