"""Limits of the 8-bit calls as include/mok.h states them, before any device work (no GPU needed)."""
import ctypes

import pytest

from test_fp8_host import BAD, OK, SMALL, UNSUPPORTED, matrix, schedule

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


TABLES = dict(counts=4, poff=5, inv=32, mblocks=4 * ((32 + 4 * 127) // 128), meta=16, row_token=32 + 4 * 127)  # int32 each


@pytest.mark.parametrize("table", TABLES)
def test_outputs_over_the_schedules_tables(mok, table):
    """A schedule's tables are inputs of the calls on routed rows: an output on the first or the last of them is refused."""
    L, s = mok._lib, schedule(mok)
    for i, k in enumerate(TABLES):
        setattr(s, k, (1 << 40) + (i << 20))
    s.topk_weights = 1 << 42
    p, at, R = ctypes.byref(s), getattr(s, table), s.rpad_max
    a = matrix(mok, rows=R, q=1 << 32, s=1 << 33)
    w = matrix(mok, rows=16, batch=4, block=True, q=1 << 34, s=1 << 35)
    t = matrix(mok, rows=24, cols=R, ld=(R + 15) // 16 * 16, q=1 << 36, s=1 << 37)
    x, far = 1 << 30, 1 << 50
    last = at + (4 * TABLES[table] - 1) // 16 * 16
    first = lambda n: at - n + 16  # noqa: E731  (its last 16 bytes on the table's first)
    tokens, rows = 16 * 64 * 2, R * 64 * 2
    for call, n in ((lambda o: L.mok_dispatch(p, x, 64, o, None), rows),
                    (lambda o: L.mok_dispatch_backward(p, x, 64, o, None), tokens),
                    (lambda o: L.mok_combine(p, x, 64, o, None), tokens),
                    (lambda o: L.mok_combine_backward(p, x, 2 * x, 64, o, far, None), rows),
                    (lambda o: L.mok_combine_backward(p, x, 2 * x, 64, far, o, None), 16 * 2 * 4),
                    (lambda o: L.mok_fp8_quantize_routed(p, 1, x, 64, o, far, None, None, None), R * 64),
                    (lambda o: L.mok_fp8_quantize_routed(p, 1, x, 64, far, o, None, None, None), R * 4),
                    (lambda o: L.mok_fp8_quantize_routed(p, 0, x, 64, None, None, o, far, None), 64 * ((R + 15) // 16 * 16)),
                    (lambda o: L.mok_fp8_quantize_routed(p, 0, x, 64, None, None, far, o, None), (R + 127) // 128 * 64 * 4),
                    (lambda o: L.mok_fp8_grouped_matmul(p, ctypes.byref(a), ctypes.byref(w), o, None), R * 16 * 2),
                    (lambda o: L.mok_fp8_grouped_wgrad(p, ctypes.byref(t), ctypes.byref(t), o, 1, None), 4 * 24 * 24 * 4)):
        assert call(first(n)) == BAD and call(last) == BAD
