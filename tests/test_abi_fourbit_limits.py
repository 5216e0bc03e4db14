"""Where the 4-bit layer's launches end, on both sides of each limit (no GPU: a call that fits stops at
its workspace, which is checked after the launches' sizes)."""
import ctypes
import os

import pytest

FAKE = ctypes.c_void_p(0x10000)
UNSUP, WS = 2, 3
INT4, MXFP4 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from grouped_gemm_histogram_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_gemm_histogram_amd.build import build
        build()
    return _lib.load()


def forward(lib, T, H, I, fmt=MXFP4, group=32, E=1, k=1):
    return lib.forward_fourbit(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, fmt, group, T, H, I, E, k, -1, 1, FAKE, 1, None,
                               FAKE, 16, None)


def rows(blocks, E=1):
    """The most rows whose blocks M/16 + E + 1 are at most `blocks`."""
    return 16 * (blocks - E - 1) + 15


@pytest.mark.parametrize("E", [1, 40])
def test_items_of_the_streaming_kernel(lib, E):
    # gate/up: 4096 columns in tiles of 8, 512 items a row block; down: 32 columns, 2
    T = rows((2 ** 31 - 1) // 512, E)
    assert forward(lib, T, 32, 4096, E=E) == WS and forward(lib, T + 1, 32, 4096, E=E) == UNSUP
    # down: 16384 columns in tiles of 16, 1024 items; gate/up: 32 columns, on rows too long to stream, 1 workgroup
    T = rows((2 ** 31 - 1) // 1024, E)
    assert forward(lib, T, 16384, 32, E=E) == WS and forward(lib, T + 1, 16384, 32, E=E) == UNSUP


def test_workgroups_of_the_long_rows_kernel(lib):
    # down: 512 columns in workgroups of 64 on rows of 7200; gate/up: 900 items a row block, within the streaming limit
    T = rows((2 ** 24 - 1) // 8)
    assert forward(lib, T, 512, 7200) == WS and forward(lib, T + 1, 512, 7200) == UNSUP
    # int4 groups of 32 stream up to 5120 channels
    T = rows((2 ** 24 - 1) // 64)
    assert forward(lib, T, 4096, 5152, INT4) == WS and forward(lib, T + 1, 4096, 5152, INT4) == UNSUP
    assert forward(lib, T + 1, 4096, 5120, INT4) == WS


def test_rows_of_a_launch(lib):
    assert forward(lib, 2 ** 31 - 65, 32, 32) == WS and forward(lib, 2 ** 31 - 64, 32, 32) == UNSUP


def test_longest_rows(lib):
    for fmt, group, K in ((INT4, 32, 16128), (INT4, 64, 32512), (INT4, 128, 65280), (MXFP4, 32, 65280)):
        assert forward(lib, 4, K, 128, fmt, group) == WS, (fmt, group)
        assert forward(lib, 4, K + max(group, 128) * 4, 128, fmt, group) == UNSUP, (fmt, group)
