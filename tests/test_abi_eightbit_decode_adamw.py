"""What the 8-bit products, the layer for few tokens and the AdamW step refuse on the host, before any launch (no GPU)."""
import ctypes
import os

import pytest

INVALID, UNSUP, WS = 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)
FAR = ctypes.c_void_p(0x40000000)
ODD = ctypes.c_void_p(0x10002)
F32, BF16, FP8 = 0, 1, 2
W_BF16, W_FP8, W_EIGHT, W_INT4, W_MXFP4 = range(5)
U32 = (1 << 32) - 1


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_histogram_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_gemm_histogram_amd.build import build
        build()
    return _lib.load()


def test_quantise_refusals(lib):
    def call(x=FAKE, xd=BF16, rows=4, H=64, codes=FAR, scales=FAKE):
        return lib.quantize_rows_eightbit(x, xd, rows, H, codes, scales, None)
    assert call(rows=0, x=None, codes=None, scales=None) == 0
    assert call(xd=FP8) == INVALID and call(rows=-1) == INVALID and call(rows=1 << 31) == INVALID
    assert call(H=0) == INVALID and call(H=24) == INVALID and call(H=32784) == UNSUP
    for name in ("x", "codes", "scales"):
        assert call(**{name: None}) == INVALID, name
    assert call(x=ODD) == INVALID and call(codes=ODD) == INVALID and call(scales=ODD) == INVALID


def product(lib, a=FAKE, sa=FAKE, rows=8, gather=None, div=1, b=FAKE, sb=FAKE, off=FAKE, E=8, M=8, N=64, K=64, epi=0,
            c=FAR, cd=BF16):
    return lib.grouped_gemm_eightbit(a, sa, rows, gather, div, b, sb, off, E, M, N, K, epi, c, cd, None)


def test_product_refusals(lib):
    assert product(lib, M=0, rows=0, a=None) == 0
    assert product(lib, E=0) == INVALID and product(lib, E=1025) == INVALID
    assert product(lib, epi=2) == INVALID and product(lib, epi=1, N=33) == INVALID
    assert product(lib, cd=FP8) == INVALID
    assert product(lib, K=24) == INVALID and product(lib, K=0) == INVALID
    assert product(lib, K=131072) == UNSUP                      # 127 * 127 * 131072 > 2^31
    assert product(lib, N=4) == INVALID and product(lib, N=4, cd=F32, E=0) == INVALID   # rows of C of 8 bytes
    assert product(lib, rows=7) == INVALID
    assert product(lib, gather=FAKE, div=0) == INVALID and product(lib, gather=FAKE, div=17) == INVALID
    assert product(lib, gather=FAKE, rows=0) == INVALID
    assert product(lib, M=1 << 26, rows=1 << 26, K=64) == INVALID and b"A must span" in lib.last_error()
    assert product(lib, N=1 << 26, K=64) == INVALID and b"B must span" in lib.last_error()
    for name in ("a", "sa", "b", "sb", "off", "c"):
        assert product(lib, **{name: None}) == INVALID, name
    for name in ("a", "b", "sb", "c", "sa"):
        assert product(lib, **{name: ODD}) == INVALID, name


def test_layer_refusals(lib):
    def call(x=FAKE, T=4, H=64, I=64, E=8, k=2, s13=FAKE, od=BF16, ws=FAKE, n=1 << 30):
        return lib.forward_eightbit(x, FAKE, FAKE, s13, FAKE, FAKE, T, H, I, E, k, -1, 1, FAR, od, None, ws, n, None)
    assert call(n=16) == WS and call(ws=None) == WS
    assert call(H=24) == INVALID and call(I=24) == INVALID and call(k=9) == INVALID and call(T=-1) == INVALID
    assert call(H=32784) == UNSUP
    assert call(x=None) == INVALID and call(s13=None) == INVALID and call(od=FP8) == INVALID
    assert lib.forward_eightbit_workspace(4, 64, 64, 8, 9) == 0
    assert lib.forward_eightbit_workspace(64, 2880, 2880, 32, 4) >= 64 * 2880 + 256 * 2880 * (2 + 1 + 2)


def decode(lib, x=FAKE, fmt=W_BF16, group=32, T=4, H=256, I=256, E=8, k=2, s=FAKE, w2=FAKE, out=FAR, od=BF16, ws=FAKE,
           n=1 << 30):
    return lib.forward_decode(x, FAKE, FAKE, s, w2, s, fmt, group, T, H, I, E, k, -1, 1, out, od, ws, n, None)


def test_few_tokens_refusals(lib):
    assert decode(lib, T=0, x=None) == 0
    assert decode(lib, T=17) == UNSUP and decode(lib, T=-1) == INVALID
    assert decode(lib, fmt=5) == INVALID and decode(lib, fmt=-1) == INVALID
    assert decode(lib, E=0) == INVALID and decode(lib, k=9) == INVALID and decode(lib, E=1025) == INVALID
    assert decode(lib, k=17, E=64) == INVALID
    for fmt, unit in ((W_BF16, 8), (W_EIGHT, 16), (W_FP8, 128), (W_MXFP4, 32)):
        assert decode(lib, fmt=fmt, H=256 + unit // 2) == INVALID
        assert decode(lib, fmt=fmt, I=256 + unit // 2) == INVALID
    for group in (32, 64, 128):
        assert decode(lib, fmt=W_INT4, group=group, I=256 + group // 2) == INVALID
    assert decode(lib, fmt=W_INT4, group=16) == INVALID and decode(lib, fmt=W_MXFP4, group=64) == INVALID
    assert decode(lib, fmt=W_INT4, H=96) == UNSUP and decode(lib, fmt=W_MXFP4, I=64) == UNSUP
    for name in ("x", "w2", "out"):
        assert decode(lib, **{name: None}) == INVALID, name
        assert decode(lib, **{name: ODD}) == INVALID, name
    assert decode(lib, fmt=W_EIGHT, s=None) == INVALID and decode(lib, fmt=W_INT4, s=ODD) == INVALID
    assert decode(lib, od=FP8) == INVALID
    assert decode(lib, n=16) == WS and decode(lib, ws=None) == WS and decode(lib, ws=ODD) == INVALID


def test_few_tokens_limits(lib):
    """The kernels' offsets: an expert's rows of one matrix, the tokens and the hidden rows stay below 2 GiB."""
    need = lib.forward_decode_workspace
    assert need(16, 7168, 2048, 256, 8) >= 16 * 8 * 2048 * 2 and need(1, 64, 64, 8, 2) > 0
    assert need(17, 64, 64, 8, 2) == 0 and need(4, 64, 64, 8, 9) == 0 and need(4, 63, 64, 8, 2) == 0
    wide = 1 << 15
    assert decode(lib, H=wide, I=wide, ws=None) == INVALID and b"4 GiB" in lib.last_error()      # 2^30 * 4 bytes
    assert decode(lib, H=wide, I=wide, fmt=W_EIGHT, ws=None) == WS                               # 2^31
    assert decode(lib, H=2 * wide, I=wide, fmt=W_EIGHT, ws=None) == INVALID
    assert decode(lib, H=2 * wide, I=wide, fmt=W_MXFP4, ws=None) == WS
    assert decode(lib, H=2 * wide, I=2 * wide, fmt=W_MXFP4, ws=None) == INVALID
    assert need(4, 2 * wide, wide, 8, 2) >= 8 * wide * 2        # a size that only some formats take
    assert decode(lib, H=(1 << 24) + 128, I=8) == UNSUP and decode(lib, I=(1 << 24) + 128, H=8) == UNSUP
    assert decode(lib, I=1 << 24, H=8, T=16, k=8) == INVALID and b"2 GiB" in lib.last_error()    # 128 rows of 32 MiB


class Hyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


def adamw(lib, n=(5, 0, 300), p=(0x10000, 0x10000, 0x11000), g=(0x20000,) * 3, pd=BF16, gd=BF16, sd=F32, m=FAKE, ms=FAKE, v=FAKE,
          vs=FAKE, master=None, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, step=1, schedule=None, gs=None, rng=None,
          hyper=True):
    from grouped_gemm_histogram_amd import _lib
    count = len(n)
    h = _lib.MoeAdamw(lr, b1, b2, eps, wd, step)
    return lib.adamw_step((ctypes.c_void_p * count)(*p), (ctypes.c_void_p * count)(*g), (ctypes.c_int64 * count)(*n),
                          count, pd, gd, sd, m, ms, v, vs, master, ctypes.byref(h) if hyper else None, schedule, gs, rng,
                          None)


def test_adamw_refusals(lib):
    assert adamw(lib, n=(0, 0, 0), p=(None,) * 3, m=None) == 0
    assert adamw(lib, hyper=False) == INVALID
    assert adamw(lib, pd=FP8) == INVALID and adamw(lib, gd=FP8) == INVALID and adamw(lib, sd=BF16) == INVALID
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan),
                dict(eps=0.0), dict(eps=nan), dict(eps=inf), dict(wd=-0.1), dict(wd=inf), dict(step=0)):
        assert adamw(lib, **bad) == INVALID, bad
    assert adamw(lib, n=(5, -1, 300)) == INVALID and adamw(lib, n=(5, (1 << 34) + 1, 300)) == INVALID
    assert adamw(lib, m=None) == INVALID and adamw(lib, v=None) == INVALID
    assert adamw(lib, sd=FP8, ms=None) == INVALID and adamw(lib, sd=FP8, vs=None) == INVALID
    assert adamw(lib, pd=F32, master=FAKE) == INVALID          # f32 params are their own copy
    for name in ("m", "v", "master", "ms", "vs", "schedule", "gs", "rng"):
        assert adamw(lib, **{name: ODD}) == INVALID, name
    assert adamw(lib, p=(0x10000, 0, 0x10000)) == INVALID and b"overlap" in lib.last_error()
    assert adamw(lib, n=(8, 0, 300), p=(0x10010, 0, 0x10000 - 512)) == INVALID and b"overlap" in lib.last_error()
    assert adamw(lib, p=(0x10000, 0, None)) == INVALID and adamw(lib, g=(None, 0, 0x10000)) == INVALID
    assert adamw(lib, p=(0x10008, 0, 0x10000)) == INVALID


def test_adamw_state_elements(lib):
    def elements(*n):
        return lib.adamw_state_elements((ctypes.c_int64 * max(len(n), 1))(*n), len(n))
    assert elements() == 0 and elements(0) == 0 and elements(1) == 128 and elements(128, 129) == 384
    assert elements(1 << 34) == 1 << 34 and elements((1 << 34) + 1) == -1 and elements(-1) == -1
    assert lib.adamw_state_elements(None, 1) == -1 and lib.adamw_state_elements(None, -1) == -1
