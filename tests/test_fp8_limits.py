"""Limits of the 8-bit calls as include/mok.h states them, before any device work (no GPU needed)."""
import ctypes

import pytest

from test_fp8_host import BAD, OK, SMALL, UNSUPPORTED, matrix

MOST = 65535 * 128  # rows that a quantisation takes


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def test_a_linear_takes_the_rows_that_its_quantisation_takes(mok):
    """No workspace is named for rows that the call then refuses, and it refuses them before it looks for one."""
    L, w = mok._lib, matrix(mok, block=True, q=1 << 60, s=1 << 61)
    f = lambda M, ws, n: L.mok_fp8_linear(1 << 20, M, ctypes.byref(w), 1 << 50, ws, n, None, None)  # noqa: E731
    size = L.mok_fp8_linear_workspace_bytes
    assert size(MOST, 64) >= MOST * 64 + 4 * MOST and f(MOST, 1 << 40, size(MOST, 64) - 1) == SMALL
    for M in (MOST + 1, MOST + 128, 2**31 - 1024):
        assert size(M, 64) == 0 and f(M, 1 << 40, 1 << 39) == UNSUPPORTED and f(M, None, 0) == UNSUPPORTED
    assert f(-1, 1 << 40, 1 << 39) == BAD and f(0, None, 0) == OK
    assert L.mok_fp8_quantize(1 << 20, MOST + 1, 64, 1 << 40, 1 << 50, None, None, None) == UNSUPPORTED
