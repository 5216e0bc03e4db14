"""What the norm, dropout and 4-bit entry points refuse on the host, before any launch (no GPU)."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUP, WS = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)
FAR = ctypes.c_void_p(0x40000000)
ODD = ctypes.c_void_p(0x10002)
F32, BF16, FP8 = 0, 1, 2
INT4, MXFP4 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_histogram_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_gemm_histogram_amd.build import build
        build()
    return _lib.load()


def norm(lib, x=FAKE, xd=BF16, T=4, H=64, w=FAKE, b=FAKE, wd=F32, eps=1e-5, rms=0, y=FAR, mean=FAKE, rstd=FAKE):
    return lib.layer_norm(x, xd, T, H, w, b, wd, eps, rms, y, mean, rstd, None)


def test_layer_norm_refusals(lib):
    assert norm(lib, T=0, x=None, y=None) == 0
    assert norm(lib, xd=FP8) == INVALID and norm(lib, wd=FP8) == INVALID
    assert norm(lib, T=-1) == INVALID and norm(lib, T=1 << 31) == INVALID and norm(lib, H=0) == INVALID
    assert norm(lib, H=32769) == UNSUP
    for eps in (-1e-5, float("nan"), float("inf")):
        assert norm(lib, eps=eps) == INVALID
    assert norm(lib, x=None) == INVALID and norm(lib, y=None) == INVALID
    assert norm(lib, x=ODD) == INVALID and norm(lib, w=ODD) == INVALID
    # y starts inside x
    assert norm(lib, y=ctypes.c_void_p(0x10010)) == INVALID
    assert b"overlaps" in lib.last_error()


def norm_bwd(lib, dy=FAKE, x=FAKE, xd=BF16, T=4, H=64, w=FAKE, wd=F32, mean=FAKE, rstd=FAKE, rms=0, dx=FAR, dw=FAKE,
             db=FAKE, gd=F32, ws=FAKE, n=1 << 30):
    return lib.layer_norm_backward(dy, x, xd, T, H, w, wd, mean, rstd, rms, dx, dw, db, gd, ws, n, None)


def test_layer_norm_backward_refusals(lib):
    assert norm_bwd(lib, xd=FP8) == INVALID and norm_bwd(lib, gd=FP8) == INVALID and norm_bwd(lib, wd=FP8) == INVALID
    assert norm_bwd(lib, H=40000) == UNSUP and norm_bwd(lib, T=-1) == INVALID
    for name in ("dy", "x", "rstd", "dx", "mean"):
        assert norm_bwd(lib, **{name: None}) == INVALID, name
    assert norm_bwd(lib, n=1) == WS and norm_bwd(lib, ws=None) == WS
    assert norm_bwd(lib, dx=ctypes.c_void_p(0x10010)) == INVALID
    assert lib.layer_norm_backward_workspace(4096, 2880) >= 2 * 2880 * 4
    assert lib.layer_norm_backward_workspace(-1, 64) == 0 and lib.layer_norm_backward_workspace(4, 40000) == 0


def drop(lib, x=FAKE, xd=BF16, r=None, rd=BF16, n=64, p=0.5, rng=FAKE, out=FAR, od=BF16):
    return lib.dropout_add(x, xd, r, rd, n, p, rng, out, od, None)


def test_dropout_refusals(lib):
    assert drop(lib, n=0, x=None, out=None) == 0
    for p in (-0.1, 1.5, float("nan")):
        assert drop(lib, p=p) == INVALID
    assert drop(lib, rng=None) == INVALID and drop(lib, rng=ODD) == INVALID
    assert drop(lib, x=None) == INVALID and drop(lib, out=None) == INVALID and drop(lib, n=-1) == INVALID
    assert drop(lib, xd=FP8) == INVALID and drop(lib, od=FP8) == INVALID and drop(lib, r=FAKE, rd=FP8) == INVALID
    assert drop(lib, out=FAKE, od=F32) == INVALID            # in place with another type
    assert drop(lib, out=ctypes.c_void_p(0x10010)) == INVALID
    assert drop(lib, x=FAR, r=FAKE, rd=F32, out=FAKE) == INVALID


def test_combine_dropout_refusals(lib):
    def call(y=FAKE, T=4, H=64, r=None, rd=BF16, p=0.1, rng=FAKE, out=FAR, od=BF16, k=2):
        return lib.unpermute_combine_dropout(y, BF16, FAKE, FAKE, FAKE, 8, T, H, k, r, rd, p, rng, out, od, None)
    assert call(T=0) == 0
    assert call(H=12) == INVALID and call(k=9) == INVALID and call(y=None) == INVALID
    assert call(p=2.0) == INVALID and call(rng=None) == INVALID and call(od=FP8) == INVALID
    assert call(r=FAR) == INVALID and b"overlaps" in lib.last_error()
    assert call(r=ODD) == INVALID and call(r=FAKE, rd=FP8) == INVALID


def matvec(lib, a=FAKE, rows=8, gather=None, div=1, codes=FAKE, scales=FAKE, fmt=INT4, group=32, off=FAKE, E=8, M=8,
           N=64, K=64, epi=0, c=FAKE, cd=BF16):
    return lib.grouped_matvec_fourbit(a, rows, gather, div, codes, scales, fmt, group, off, E, M, N, K, epi, c, cd,
                                      None)


def test_fourbit_refusals(lib):
    assert matvec(lib, M=0, rows=0, a=None) == 0
    assert matvec(lib, E=0) == INVALID and matvec(lib, E=1025) == INVALID
    assert matvec(lib, fmt=2) == INVALID and matvec(lib, fmt=MXFP4, group=64) == INVALID
    assert matvec(lib, group=48) == INVALID and matvec(lib, group=128) == INVALID     # K = 64
    assert matvec(lib, K=72) == INVALID and matvec(lib, K=0) == INVALID
    assert matvec(lib, epi=2) == INVALID and matvec(lib, epi=1, N=63) == INVALID
    assert matvec(lib, cd=FP8) == INVALID
    assert matvec(lib, rows=7) == INVALID                     # fewer rows of A than of the product
    assert matvec(lib, gather=FAKE, div=0) == INVALID and matvec(lib, gather=FAKE, div=17) == INVALID
    assert matvec(lib, gather=FAKE, rows=0) == INVALID
    for name in ("a", "codes", "scales", "off", "c"):
        assert matvec(lib, **{name: None}) == INVALID, name
    assert matvec(lib, a=ODD) == INVALID and matvec(lib, codes=ODD) == INVALID
    assert matvec(lib, M=1 << 30, rows=1 << 30, N=1 << 20) == UNSUP
    assert matvec(lib, M=(1 << 31) - 1, rows=(1 << 31) - 1) == UNSUP

    q = lambda wd=BF16, E=2, N=4, K=64, fmt=INT4, group=32, w=FAKE: lib.quantize_fourbit(
        w, wd, E, N, K, fmt, group, FAKE, FAKE, None)
    assert q(wd=FP8) == INVALID and q(E=0) == INVALID and q(K=48) == INVALID and q(w=None) == INVALID
    assert q(fmt=MXFP4, group=128, K=128) == INVALID and q(N=1 << 30, K=1 << 20) == INVALID

    fwd = lambda T=4, H=64, I=64, E=8, k=2, group=32, ws=FAKE, n=1 << 30, x=FAKE, od=BF16: lib.forward_fourbit(
        x, FAKE, FAKE, FAKE, FAKE, FAKE, INT4, group, T, H, I, E, k, -1, 1, FAKE, od, None, ws, n, None)
    assert fwd(n=16) == WS and fwd(ws=None) == WS
    assert fwd(H=48) == INVALID and fwd(I=48) == INVALID and fwd(group=128) == INVALID and fwd(k=9) == INVALID
    assert fwd(x=None) == INVALID and fwd(od=FP8) == INVALID and fwd(T=-1) == INVALID
    assert lib.forward_fourbit_workspace(4, 64, 64, 8, 9) == 0
    assert lib.forward_fourbit_workspace(64, 2880, 2880, 32, 4) >= 2 * 256 * 2880 * 2


def test_wrappers_refuse_cpu_tensors():
    import grouped_gemm_histogram_amd as g
    x = torch.zeros(4, 64)
    for call in (lambda: g.layer_norm(x), lambda: g.dropout_add(x, torch.zeros(2, dtype=torch.int64), 0.5),
                 lambda: g.quantize_fourbit(x[None]),
                 lambda: g.layer_norm_backward(x, x, g.NormStats(None, torch.zeros(4)))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
