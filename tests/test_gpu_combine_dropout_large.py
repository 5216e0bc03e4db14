"""Combine with dropout on expert rows past 256 MiB, where four column steps are in flight, with each type of
residual, against the same steps apart: the plain combine's f32 sums, then dropout with the residual."""
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("ydt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rdt", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_combine_dropout_past_256_mib(ydt, rdt, odt):
    import grouped_gemm_histogram_amd as g
    T, k, H, E = 9001, 4, 4096, 16                     # 295 MB of bf16 rows, 590 of f32
    say(f"unpermute_combine_dropout T={T} H={H} {ydt} {rdt} {odt}")
    gen = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)
    ids, w = g.route_topk(rand(T, E), k, T * k - 1001)
    offsets, _, row_pos = g.build_offsets(ids, E)
    y = rand(T * k, H).to(ydt)
    y[T * k - 1001:] = float("nan")                    # rows without an expert are never read
    r = None if rdt is None else rand(T, H).to(rdt)
    rng = torch.tensor([21, (1 << 32) - 2], dtype=torch.int64, device=DEV)
    out = g.unpermute_combine_dropout(y, row_pos, w, offsets, k, rng, 0.3, residual=r, out_dtype=odt)
    sums = g.unpermute_combine(y, row_pos, w, offsets, k, out_dtype=torch.float32)
    want = g.dropout_add(sums, rng, 0.3, residual=r, out_dtype=odt)
    assert out.dtype == odt and torch.equal(out, want)
    # the sums themselves, on some tokens, in 64 bits: k products and additions
    at = torch.arange(0, T, 97, device=DEV)
    pos = row_pos.view(T, k)[at].long()
    wt = (w.view(T, k)[at] * (pos < offsets[-1])).double()
    rows = torch.where((pos < offsets[-1])[..., None], y[pos].double(), 0.0)
    ref, mag = (rows * wt[..., None]).sum(1), (rows * wt[..., None]).abs().sum(1)
    assert bool(((sums[at].double() - ref).abs() <= 2 * k * 2.0 ** -24 * mag).all())
