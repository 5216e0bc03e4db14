"""What the f32 sums of int4 products hold, on inputs whose sums are whole numbers.

A sum of whole numbers is exact in f32, in any order, while no partial sum passes 2^24.  With codes 0 to 15
and the offset -8 taken apart, partial sums are at most (15 + 8) * scale * sum |a|.
"""
import numpy as np
import pytest
import torch

from helpers import say
from oracle import fourbit as ofb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def product(a, codes, scales, off):
    import grouped_gemm_histogram_amd as g
    out = g.grouped_matvec_fourbit(a.to(DEV), codes.to(DEV), scales.to(DEV),
                                   torch.tensor(off, dtype=torch.int32, device=DEV), out_dtype=torch.float32)
    return out.cpu().double().numpy()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [512, 2048, 7296])     # streaming with one and two steps a wave, and the long rows' kernel
def test_int4_sums_of_large_and_small_activations(group, K):
    """Four runs of 32 channels with 18 activations up to 8160 and 14 odd ones up to 255: a run's sum |a| is
    at most 150450, and 23 * 4 * 150450 < 2^24; a run's sum of 136 |a| passes 2^24."""
    gen = torch.Generator().manual_seed(group + K)
    M, N, off = 21, 50, [0, 17, 21]
    codes = torch.randint(0, 256, (2, N, K // 2), generator=gen, dtype=torch.uint8)
    scales = torch.ones(2, N, K // group)
    a = torch.zeros(M, K)
    runs = torch.randperm(K // 32, generator=gen)[:4]
    for r in runs.tolist():
        at = r * 32 + torch.randperm(32, generator=gen)
        a[:, at[:18]] = 32.0 * torch.randint(200, 256, (M, 18), generator=gen).float()
        a[:, at[18:]] = 2.0 * torch.randint(0, 128, (M, 14), generator=gen).float() + 1.0
    assert 23 * float(a.sum(1).max()) < 2 ** 24
    a16 = a.to(torch.bfloat16)
    assert torch.equal(a16.float(), a)
    say(f"int4 sums, groups of {group}, K={K}")
    got = product(a16, codes, scales, off)
    for e in range(2):
        rows = slice(off[e], off[e + 1])
        np.testing.assert_array_equal(got[rows], a[rows].double().numpy() @
                                      ofb.dequantize(codes[e].numpy(), scales[e].numpy()).T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [256, 2048, 7296])
def test_int4_largest_activations(group, K):
    """Every activation 2^117, the documented limit of a group of 128: 15 * 128 * 2^117 = 1.875 * 2^127.  With
    scales of 2^-100 each partial sum is 2^17 times a whole number of at most 23 * 7296 < 2^24: exact."""
    N = 20
    gen = torch.Generator().manual_seed(group)
    codes = torch.randint(0, 256, (1, N, K // 2), generator=gen, dtype=torch.uint8)
    codes[0, 0], codes[0, 1] = 0, 255                     # every weight -8, every weight 7
    scales = torch.full((1, N, K // group), 2.0 ** -100)
    a = torch.full((3, K), 2.0 ** 117, dtype=torch.bfloat16)
    a[1] = -a[1]
    say(f"int4 largest activations, groups of {group}, K={K}")
    got = product(a, codes, scales, [0, 3])
    np.testing.assert_array_equal(got, a.double().numpy() @ ofb.dequantize(codes[0].numpy(), scales[0].numpy()).T)


@pytest.mark.parametrize("fmt,group", [("mxfp4", 32), ("int4", 32), ("int4", 128)])
@pytest.mark.parametrize("K", [512, 7296])
def test_rows_beside_infinite_and_nan_rows(fmt, group, K):
    """A row with an infinity or NaN is not finite; the rows beside it keep their bits."""
    import grouped_gemm_histogram_amd as g
    gen = torch.Generator().manual_seed(3)
    N = 24
    codes = torch.randint(0, 256, (1, N, K // 2), generator=gen, dtype=torch.uint8).to(DEV)
    if fmt == "mxfp4":
        scales = torch.randint(118, 124, (1, N, K // 32), generator=gen, dtype=torch.uint8).to(DEV)
    else:
        scales = torch.rand(1, N, K // group, generator=gen).to(DEV)
    a = torch.randn(20, K, generator=gen).to(torch.bfloat16).to(DEV)
    off = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    want = g.grouped_matvec_fourbit(a, codes, scales, off)
    b = a.clone()
    b[2, 5], b[18, K - 1], b[19, 0] = float("nan"), float("inf"), -float("inf")
    got = g.grouped_matvec_fourbit(b, codes, scales, off)
    bad = torch.zeros(20, dtype=torch.bool, device=DEV)
    bad[[2, 18, 19]] = True
    assert torch.equal(got[~bad], want[~bad])
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[18:]).any()
