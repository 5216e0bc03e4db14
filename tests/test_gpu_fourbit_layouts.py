"""4-bit products over every layout of their kernels: each count of 128-channel steps a wave holds when
streaming (one to seven of 1024 channels), both sides of the step to the long rows' kernel, more items
a workgroup than the ring has slots, and inexact data on long rows.

References are in 64 bits on the GPU from elementary operations.  Tolerances of inexact data (u = 2^-24): mxfp4
operands are exact, so a sum of K terms is off by at most 2 K u of sum |a w| (2 u an addition also covers an
accumulator that truncates).  int4 sums codes 0 to 15 and the offset 8, (15 + 8) |a| a channel, over a group, and
scales: at most 2 (2 group + 2 + K / 32) u * 23 * |scale| * sum |a|.
"""
import pytest
import torch

from helpers import say
from oracle import fourbit as ofb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
FORMATS = [("mxfp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)]


def weights(E, N, K, fmt, group, seed, exact):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
    if fmt == "mxfp4":
        lo, hi = (126, 129) if exact else (110, 125)
        return codes, torch.randint(lo, hi, (E, N, K // 32), generator=gen, device=DEV, dtype=torch.uint8)
    if exact:
        return codes, 2.0 ** torch.randint(-1, 2, (E, N, K // group), generator=gen, device=DEV).float()
    return codes, 0.01 * (0.5 + torch.rand(E, N, K // group, generator=gen, device=DEV))


def values(codes, scales):
    """float64 weights [N, K] and scales [N, K] of one expert."""
    N, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], 2).view(N, 2 * half).long()
    if scales.dtype == torch.uint8:
        v, s = torch.from_numpy(ofb.E2M1).to(DEV)[c], torch.exp2(scales.double() - 127.0)
    else:
        v, s = c.double() - 8.0, scales.double()
    s = s.repeat_interleave(2 * half // scales.shape[1], 1)
    return v * s, s


def reference(a, codes, scales, off, silu, exact):
    """(result, tolerance of an f32 result) for permuted rows a [M, K]."""
    E, N, K = codes.shape[0], codes.shape[1], a.shape[1]
    group = K // scales.shape[2]
    n_out = N // 2 if silu else N
    ref = torch.zeros(a.shape[0], n_out, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(ref)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        x = a[lo:hi].double()
        w, s = values(codes[e], scales[e])
        acc = torch.mm(x, w.t().contiguous())
        if exact:
            err = torch.zeros_like(acc)
        elif scales.dtype == torch.uint8:
            err = 2 * K * U * torch.mm(x.abs(), w.abs().t().contiguous())
        else:
            err = 2 * (2 * group + 2 + K / 32) * U * 23 * torch.mm(x.abs(), s.abs().t().contiguous())
        if silu:
            gate, up = acc[:, :n_out], acc[:, n_out:]
            sg = gate / (1 + torch.exp(-gate))
            # SiLU's slope is at most 1.1; its own rounding: 8 u, and 1.5 u |gate| of the exponential's argument
            t = 1.1 * up.abs() * err[:, :n_out] + sg.abs() * err[:, n_out:] + 1.1 * err[:, :n_out] * err[:, n_out:]
            tol[lo:hi] = t + (8 * U + 1.5 * U * gate.abs()) * (sg * up).abs() + 2.0 ** -121 * up.abs()
            acc = sg * up
        else:
            tol[lo:hi] = err + U * acc.abs()
        ref[lo:hi] = acc
    return ref, tol


def run(a, codes, scales, off, silu, **kw):
    import grouped_gemm_histogram_amd as g
    return g.grouped_matvec_fourbit(a, codes, scales, torch.tensor(off, dtype=torch.int32, device=DEV),
                                    "silu_mul" if silu else "none", **kw)


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1024, 1024 + 32, 2048, 3000, 4096, 4096 + 32, 5120, 5120 + 32, 6100, 6144, 7168, 7168 + 32])
def test_steps_and_items(fmt, group, silu, K):
    """Small whole activations and power-of-two scales: every sum is exact (23 * 2 * 2 * 7296 < 2^24 halves).  Ten
    blocks of rows by 513 tiles of columns (the last one partial) are 10 to 21 items a workgroup."""
    K = -(-K // group) * group
    off, M, N = [0, 100, 100, 137], 140, 8200
    say(f"steps {fmt} {group} silu={silu} K={K}")
    codes, scales = weights(3, N, K, fmt, group, K, True)
    gen = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randint(-2, 3, (M, K), generator=gen, device=DEV).to(torch.bfloat16)
    ref, tol = reference(a, codes, scales, off, silu, True)
    out = torch.full((M, ref.shape[1]), float("nan"), device=DEV)
    run(a, codes, scales, off, silu, out=out)
    if silu:
        assert bool(((out.double() - ref).abs() <= tol).all())
    else:
        assert torch.equal(out.double(), ref)
    assert bool((out[137:] == 0).all())


@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("K", [1536, 4992, 6144, 7424, 14336])
def test_inexact_data(fmt, group, silu, K):
    """Random activations around 0 and around 1, f32 and bf16 results."""
    off, M, N = [0, 1, 18, 18, 51], 53, 258
    for mean in (0.0, 1.0):
        say(f"inexact {fmt} {group} silu={silu} K={K} mean={mean}")
        codes, scales = weights(4, N, K, fmt, group, K + 1, False)
        gen = torch.Generator(device=DEV).manual_seed(6)
        a = (torch.randn(M, K, generator=gen, device=DEV) + mean).to(torch.bfloat16)
        ref, tol = reference(a, codes, scales, off, silu, False)
        out = run(a, codes, scales, off, silu, out_dtype=torch.float32)
        assert bool(((out.double() - ref).abs() <= tol).all())
        assert torch.equal(run(a, codes, scales, off, silu), out.to(torch.bfloat16))


@pytest.mark.parametrize("K", [2048, 7424])
def test_two_streams_at_once(K):
    """Two products on two streams, each with inputs of its own, repeatedly: each as alone."""
    off, M, N = [0, 40, 40, 57], 60, 4096
    work = []
    for i, (fmt, group) in enumerate((("int4", 128), ("mxfp4", 32))):
        codes, scales = weights(3, N, K, fmt, group, i, False)
        gen = torch.Generator(device=DEV).manual_seed(20 + i)
        a = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16)
        work.append((a, codes, scales, off, bool(i)))
    want = [run(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for rep in range(4):
        got = []
        for w, s in zip(work, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append([run(*w) for _ in range(3)])
        torch.cuda.synchronize()
        for outs, ref in zip(got, want):
            assert all(torch.equal(o, ref) for o in outs), f"repetition {rep}"


def test_same_bits_every_run():
    """A call's result does not vary, whatever ran between."""
    off, M = [0, 100, 137], 137
    for fmt, group in FORMATS:
        for K in (2048, 7424):
            codes, scales = weights(2, 2050, K, fmt, group, 1, False)
            gen = torch.Generator(device=DEV).manual_seed(2)
            a = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16)
            want = run(a, codes, scales, off, True, out_dtype=torch.float32)
            other = torch.randn_like(a)
            for _ in range(5):
                run(other, codes, scales, off, False)
                assert torch.equal(run(a, codes, scales, off, True, out_dtype=torch.float32), want), (fmt, group, K)


@pytest.mark.parametrize("E", [63, 64, 65, 129, 1000, 1024])
@pytest.mark.parametrize("K", [64, 7424])
def test_many_experts(E, K):
    """Up to sixteen experts a lane of the scan, many of them without rows."""
    gen = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 40, (E,), generator=gen) * (torch.rand(E, generator=gen) < 0.3)
    counts[0], counts[-1] = 0, 17
    off = [0] + torch.cumsum(counts, 0).tolist()
    M, N = off[-1] + 5, 24
    say(f"many experts E={E} K={K} rows={M}")
    for fmt, group in (("mxfp4", 32), ("int4", 64)):
        codes, scales = weights(E, N, K, fmt, group, E, True)
        a = torch.randint(-2, 3, (M, K), generator=gen).to(torch.bfloat16).to(DEV)
        ref, _ = reference(a, codes, scales, off, False, True)
        out = torch.full((M, N), float("nan"), device=DEV)
        run(a, codes, scales, off, False, out=out)
        assert torch.equal(out.double(), ref)
