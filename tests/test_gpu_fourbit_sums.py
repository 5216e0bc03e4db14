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
