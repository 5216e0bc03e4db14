"""The layer for few tokens on the GPU against the float64 oracle, in every weight format.

Tolerance (u = 2^-24), for one token, with |.| of every term.  A sum of K products of bf16 values (exact in f32): at
most K u of the sum of magnitudes, 2 K u to cover an accumulator that truncates; int4 sums code * x
and 8 * x, up to 23 |x| where the weight has at least 0, so 23 * scale * |x| stands for its magnitudes; a scale's
product and the joining of shares: 40 u more.  SiLU * up as in test_gpu_eightbit: 1.1 |up| for an absolute error
of the gate, |silu(gate)| for up's, (8 + 1.5 |gate|) u of itself, 2^-121 |up|.  h is then rounded to bf16: 2^-9 of
it (half a step, eps / 2 = 2^-8 relative to a value at the low end of its binade; 2^-8 is taken).  The down product
passes on h's error by |W2| and adds its own; the weights (a softmax: below 16 u) and the sum over
k terms: 2 k + 20 u.  A bf16 output: 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, row_rel_err, say
from oracle import e4m3, eightbit as o8, fourbit as ofb, routing

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FORMATS = ["bf16", "fp8", "int8", "int4/32", "int4/64", "int4/128", "mxfp4"]
UNIT = {"bf16": 8, "fp8": 128, "int8": 16, "int4/32": 32, "int4/64": 64, "int4/128": 128, "mxfp4": 32}


def make(E, N, K, fmt, seed):
    """(weights, scales on the host, values [E, N, K] in float64, magnitudes that a sum may pass through)."""
    r = np.random.default_rng(seed)
    v = (r.normal(size=(E, N, K)) / K ** 0.5).astype(np.float32)
    if fmt == "bf16":
        w = torch.from_numpy(v).to(torch.bfloat16)
        val = w.double().numpy()
        return w, None, val, np.abs(val)
    if fmt == "int8":
        c, s = o8.quantize_rows(v)
        c[:, ::3, 0] = -128                        # the code that the quantiser does not make
        val = c.astype(np.float64) * s[..., None]
        return torch.from_numpy(c), torch.from_numpy(s), val, np.abs(val)
    if fmt == "fp8":
        s = (np.abs(v).reshape(E, N // 128, 128, K // 128, 128).max(axis=(2, 4)) / 448).astype(np.float32)
        big = np.repeat(np.repeat(s, 128, 1), 128, 2)
        c = e4m3.encode(v / big)
        val = e4m3.decode(c) * big
        return torch.from_numpy(c).view(torch.float8_e4m3fn), torch.from_numpy(s), val, np.abs(val)
    group = 32 if fmt == "mxfp4" else int(fmt.split("/")[1])
    c = torch.from_numpy(r.integers(0, 256, (E, N, K // 2)).astype(np.uint8))
    if fmt == "mxfp4":
        s = torch.from_numpy(r.integers(118, 124, (E, N, K // 32)).astype(np.uint8))
        val = ofb.dequantize(c.numpy(), s.numpy())
        return c, s, val, np.abs(val)
    s = torch.from_numpy((0.02 * (0.2 + r.random((E, N, K // group)))).astype(np.float32))
    val = ofb.dequantize(c.numpy(), s.numpy())
    return c, s, val, 23 * np.repeat(s.double().numpy(), group, axis=2)


class Case:
    def __init__(self, fmt, T, H, I, E, k, seed=0, spread=True):
        r = np.random.default_rng(seed + 1000)
        self.fmt, self.k = fmt, k
        self.x = torch.from_numpy(r.normal(size=(T, H)).astype(np.float32)).to(torch.bfloat16)
        logits = r.normal(size=(T, E)).astype(np.float32)
        if not spread:
            logits += np.linspace(8, 0, E, dtype=np.float32)   # all tokens to the first experts
        self.logits = logits
        self.w13, self.s13, self.v13, self.m13 = make(E, 2 * I, H, fmt, seed)
        self.w2, self.s2, self.v2, self.m2 = make(E, H, I, fmt, seed + 1)

    def on_gpu(self):
        to = lambda t: None if t is None else t.to(DEV)
        return (to(self.x), torch.from_numpy(self.logits).to(DEV), to(self.w13), to(self.w2), self.k), \
            dict(w13_scale=to(self.s13), w2_scale=to(self.s2))

    def run(self, **more):
        args, scales = self.on_gpu()
        return g.forward_decode(*args, **scales, **more)

    def reference(self, valid=-1, renormalize=True, out=torch.bfloat16):
        x = self.x.double().numpy()
        T, H = x.shape
        E, I2, _ = self.v13.shape
        I = I2 // 2
        ids, w = routing.route_topk(self.logits, self.k, valid, renormalize)
        ids, w = np.asarray(ids).reshape(T, self.k), np.asarray(w, np.float64).reshape(T, self.k)
        ref, tol = np.zeros((T, H)), np.zeros((T, H))
        for t in range(T):
            total = np.zeros(H)
            for j in range(self.k):
                e = int(ids[t, j])
                if e == E:
                    continue
                acc = self.v13[e] @ x[t]
                err = (2 * H + 40) * U * (self.m13[e] @ np.abs(x[t]))
                gate, up = acc[:I], acc[I:]
                silu = gate / (1 + np.exp(-gate))
                h = silu * up
                eh = 1.1 * np.abs(up) * err[:I] + (np.abs(silu) + 1.1 * err[:I]) * err[I:]
                eh = eh + np.abs(h) * (8 + 1.5 * np.abs(gate)) * U + 2.0 ** -121 * np.abs(up)
                eh = eh + 2.0 ** -8 * np.abs(h)
                y = self.v2[e] @ h
                ey = np.abs(self.v2[e]) @ eh + (2 * I + 40) * U * (self.m2[e] @ (np.abs(h) + eh))
                ref[t] += w[t, j] * y
                tol[t] += w[t, j] * ey
                total += w[t, j] * np.abs(y)
            tol[t] += (2 * self.k + 20) * U * total
        if out == torch.bfloat16:
            tol += 2.0 ** -8 * (np.abs(ref) + tol)
        return ref, tol

    def check(self, valid=-1, renormalize=True, out=torch.bfloat16):
        got = self.run(num_valid_rows=valid, renormalize=renormalize, out_dtype=out)
        ref, tol = self.reference(valid, renormalize, out)
        bad = np.abs(np32(got).astype(np.float64) - ref) > tol
        say("  largest error / tolerance", float((np.abs(np32(got) - ref) / np.maximum(tol, 1e-300))[tol > 0].max())
            if (tol > 0).any() else 0.0)
        assert not bad.any(), int(bad.sum())
        return got, ref


# T, H, I, E, k, valid rows (-1: all), in units of the format
SIZES = [(1, 1, 1, 1, 1, -1), (1, 3, 5, 8, 2, -1), (16, 5, 3, 4, 2, -1), (16, 2, 2, 40, 8, 101), (5, 4, 7, 130, 3, 11),
         (7, 3, 2, 300, 16, -1), (16, 1, 1, 16, 16, 1), (16, 3, 1, 16, 16, -1), (3, 2, 3, 5, 5, 0), (12, 9, 4, 3, 1, 12)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,I,E,k,valid", SIZES)
def test_sizes(fmt, T, H, I, E, k, valid):
    u = UNIT[fmt]
    if u == 128 and E > 40:
        E = 20                                     # the host's products
        k = min(k, E)
    H, I = H * u, I * u
    if "4" in fmt:                                 # 4-bit rows have at least 128 channels
        H, I = max(H, 128), max(I, 128)
    say("decode", fmt, T, H, I, E, k, valid)
    c = Case(fmt, T, H, I, E, k, seed=T * 31 + E)
    got, ref = c.check(valid, renormalize=T != 5, out=torch.float32 if T % 2 else torch.bfloat16)
    assert (np32(got)[np.abs(ref).sum(axis=1) == 0] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_rows_and_all_tokens_on_the_same_experts(fmt):
    """Rows of more pieces than waves hold at once, ends inside a piece; sixteen rows for each of two experts."""
    u = UNIT[fmt]
    say("decode long", fmt)
    H, I = -(-2080 // u) * u, -(-1200 // u) * u
    Case(fmt, 16, H, I, 3, 2, seed=5, spread=False).check(out=torch.float32)
    Case(fmt, 2, I, H, 4, 3, seed=6).check(valid=4)


def test_same_routing_and_values_as_the_layer():
    """bf16: the result differs from the layer's by the roundings of its expert outputs."""
    c = Case("bf16", 9, 256, 192, 32, 4, seed=3)
    args, _ = c.on_gpu()
    a, b = c.run(num_valid_rows=30), g.forward(*args, num_valid_rows=30)
    assert row_rel_err(np32(a), np32(b)) < 1e-2


def test_ties_go_to_the_lower_expert():
    c = Case("bf16", 4, 64, 64, 8, 3, seed=4)
    c.logits[:] = 1.0
    c.logits[1, 5] = 2.0
    c.check()


def test_a_bad_weight_or_token_stays_with_its_tokens():
    c = Case("bf16", 6, 64, 64, 16, 2, seed=8)
    ids, _ = routing.route_topk(c.logits, 2)
    ids = np.asarray(ids).reshape(6, 2)
    clean = np32(c.run())
    c.x[2, 7] = float("nan")
    got = np32(c.run())
    assert np.isnan(got[2]).all() and (np.delete(got, 2, 0) == np.delete(clean, 2, 0)).all()
    c = Case("bf16", 6, 64, 64, 16, 2, seed=8)
    e = int(ids[3, 1])
    c.w2[e, 5, 60] = float("inf")
    got = np32(c.run())
    hit = (ids == e).any(axis=1)
    assert not np.isfinite(got[hit, 5]).any() and (got[~hit] == clean[~hit]).all()
    assert (np.delete(got, 5, 1) == np.delete(clean, 5, 1)).all()


@pytest.mark.parametrize("fmt", ["bf16", "int4/32"])
def test_the_same_bits_every_time(fmt):
    c = Case(fmt, 16, 512, 256, 16, 4, seed=9)
    args, scales = c.on_gpu()
    first = g.forward_decode(*args, **scales)
    for _ in range(20):
        assert torch.equal(first, g.forward_decode(*args, **scales))


def test_a_token_alone_and_among_others():
    """A token's result does not depend on the others but for where its sums are split."""
    c = Case("int8", 16, 256, 128, 8, 2, seed=10)
    args, scales = c.on_gpu()
    x, logits, w13, w2, k = args
    both = g.forward_decode(*args, **scales, out_dtype=torch.float32)
    for t in (0, 7, 15):
        one = g.forward_decode(x[t:t + 1].clone(), logits[t:t + 1].clone(), w13, w2, k, **scales, out_dtype=torch.float32)
        assert row_rel_err(np32(one), np32(both)[t:t + 1]) < 2.0 ** -7


def test_workspaces_streams_and_a_replayed_graph():
    c = Case("mxfp4", 8, 256, 128, 16, 4, seed=11)
    args, scales = c.on_gpu()
    want = g.forward_decode(*args, **scales)
    need = g.forward_decode_workspace_bytes(8, 256, 128, 16, 4)
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    call = lambda: g.forward_decode(*args, **scales, out=out, workspace=ws[:need])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and bool((ws[need:] == 255).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        out.zero_()
        ws.random_(0, 256)
        if i:
            args[0].copy_(torch.randn(args[0].shape, device=DEV))
            args[1].copy_(torch.randn(args[1].shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g.forward_decode(*args, **scales))


def test_two_calls_at_once():
    a, b = Case("bf16", 4, 512, 256, 8, 2, seed=12), Case("fp8", 16, 512, 256, 8, 2, seed=13)
    (aa, sa), (ab, sb) = a.on_gpu(), b.on_gpu()
    wa, wb = g.forward_decode(*aa, **sa), g.forward_decode(*ab, **sb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        with torch.cuda.stream(s1):
            ra = g.forward_decode(*aa, **sa)
        with torch.cuda.stream(s2):
            rb = g.forward_decode(*ab, **sb)
        torch.cuda.synchronize()
        assert torch.equal(ra, wa) and torch.equal(rb, wb)


def test_empty_and_refused():
    f = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)
    lg = lambda *s: torch.zeros(*s, device=DEV)
    assert g.forward_decode(f(0, 16), lg(0, 4), f(4, 32, 16), f(4, 16, 16), 2).shape == (0, 16)
    with pytest.raises(RuntimeError, match="few tokens"):
        g.forward_decode(f(17, 16), lg(17, 4), f(4, 32, 16), f(4, 16, 16), 2)
    with pytest.raises(RuntimeError, match="multiples"):
        g.forward_decode(f(1, 12), lg(1, 4), f(4, 32, 12), f(4, 12, 16), 2)
    with pytest.raises(RuntimeError):
        g.forward_decode(f(1, 16), lg(1, 4), f(4, 32, 16), f(4, 16, 16), 5)
    with pytest.raises(RuntimeError, match="workspace"):
        g.forward_decode(f(1, 16), lg(1, 4), f(4, 32, 16), f(4, 16, 16), 2,
                         workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        g.forward_decode(f(1, 16), lg(1, 5), f(4, 32, 16), f(4, 16, 16), 2)
    with pytest.raises(ValueError):
        g.forward_decode(f(1, 16), lg(1, 4), f(4, 32, 16), f(4, 16, 24), 2)
    with pytest.raises(ValueError):
        g.forward_decode(f(1, 16), lg(1, 4), f(4, 32, 16), f(4, 16, 16), 2, w13_scale=lg(4, 32), w2_scale=lg(4, 16))
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError, match="128 channels"):
        g.forward_decode(f(1, 96), lg(1, 4), u8(4, 256, 48), u8(4, 96, 64), 2, w13_scale=u8(4, 256, 3), w2_scale=u8(4, 96, 4))
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)
    with pytest.raises(ValueError):
        g.forward_decode(f(1, 16), lg(1, 4), i8(4, 32, 16), i8(4, 16, 16), 2)
    with pytest.raises(ValueError):
        g.forward_decode(f(1, 16), lg(1, 4), i8(4, 32, 16), i8(4, 16, 16), 2, w13_scale=lg(4, 33), w2_scale=lg(4, 16))
