"""Refusals of the routed-row and 8-bit calls, of the library and of the binding, before any device work (no GPU needed)."""
import ctypes

import pytest
import torch

from test_devices import _tensors
from test_streams import _Streams

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
OK, BAD, UNSUPPORTED, SMALL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def matrix(mok, rows=32, cols=64, ld=64, batch=1, block=False, q=256, s=256):
    return mok.mok_fp8_matrix(q, s, rows, cols, ld, batch, int(block))


def schedule(mok, T=16, E=4, K=2):
    """A schedule's host struct with tables at made-up addresses."""
    s = mok.mok_schedule()
    s.shape, s.config = mok.make_shape(T, 128, 128, E, K), mok.make_config(256, 2048)
    s.rpad_max = T * K + 127 * E
    s.mblocks_max = s.rpad_max // 128
    for k in ("counts", "poff", "inv", "mblocks", "meta", "row_token", "topk_weights"):
        setattr(s, k, 256)
    return s


def test_products(mok):
    f = lambda a, b, out=256, dt=0: mok._lib.mok_fp8_matmul(ctypes.byref(a), ctypes.byref(b), out, dt, None, None)  # noqa: E731
    m = lambda **k: matrix(mok, **k)  # noqa: E731
    good = m()
    for a in (m(ld=40), m(ld=48), m(cols=80, ld=64), m(rows=-1), m(cols=-8), m(batch=2), m(block=True), m(q=8), m(q=None), m(s=4),
              m(s=None), m(rows=2**31), m(cols=2**31, ld=2**31)):
        assert f(a, good) == BAD
    for b in (m(cols=48), m(rows=12), m(rows=0), m(batch=2), m(q=264)):
        assert f(good, b) == BAD
    a = m()
    a.scaling = 2
    assert f(a, good) == BAD and f(good, a) == BAD
    assert f(good, good, dt=2) == BAD and f(good, good, out=None) == BAD and f(good, good, out=264) == BAD
    assert mok._lib.mok_fp8_matmul(None, ctypes.byref(good), 256, 0, None, None) == BAD
    assert f(m(rows=0), good) == OK  # nothing to do
    b = m(q=1 << 20, s=2 << 20)
    for out in (256, 256 + 32 * 64 - 16, (1 << 20) + 16, (2 << 20) - 16):  # over a's codes, their end, b's codes, b's scales
        assert f(m(q=256, s=4096), b, out=out, dt=1) == BAD


def test_linear(mok):
    w = matrix(mok, block=True)
    f = lambda x, M, w, out, ws, n: mok._lib.mok_fp8_linear(x, M, ctypes.byref(w), out, ws, n, None, None)  # noqa: E731
    size = mok._lib.mok_fp8_linear_workspace_bytes
    assert size(100, 64) >= 100 * 64 + 4 * 100 and size(8, 64) == 256 and size(2**31, 64) == 0 and size(5, 60) == 0
    assert f(256, 100, matrix(mok), 256, 256, 1 << 20) == BAD  # scales per row
    assert f(256, 100, matrix(mok, cols=60, block=True), 256, 256, 1 << 20) == BAD
    assert f(None, 100, w, 256, 256, 1 << 20) == BAD and f(256, 100, w, 264, 256, 1 << 20) == BAD
    assert f(256, 100, w, 256, None, 1 << 20) == BAD and f(256, 100, w, 256, 272, 1 << 20) == BAD
    assert f(256, 100, matrix(mok, block=True, q=1 << 22, s=1 << 23), 1 << 24, 256, size(100, 64) - 1) == SMALL
    assert f(256, 4, w, 256, 256, 1 << 20) == BAD and f(256, 4, w, 256 + 4 * 128 - 16, 256, 1 << 20) == BAD  # out over x
    assert f(256, -1, w, 256, 256, 1 << 20) == BAD and f(None, 0, w, None, None, 0) == OK


def test_quantisation(mok):
    q = mok._lib.mok_fp8_quantize
    assert q(256, 4, 12, 256, 256, None, None, None) == BAD and q(256, 4, 0, 256, 256, None, None, None) == BAD
    assert q(256, -1, 64, 256, 256, None, None, None) == BAD and q(264, 4, 64, 256, 256, None, None, None) == BAD
    assert q(256, 4, 64, None, None, None, None, None) == BAD  # nothing asked for
    assert q(256, 4, 64, 256, None, None, None, None) == BAD and q(256, 4, 64, 256, 256, 256, None, None) == BAD
    assert q(256, 4, 64, 256, 260, None, None, None) == BAD
    assert q(256, 65535 * 128 + 1, 64, 256, 256, None, None, None) == UNSUPPORTED
    assert q(None, 0, 64, None, None, None, None, None) == OK
    assert q(256, 4, 64, 512, 8192, None, None, None) == BAD and q(256, 4, 64, None, None, 256 + 496, 8192, None) == BAD  # over x
    b = mok._lib.mok_fp8_quantize_blocks
    for batch, rows, cols in ((0, 64, 64), (1, 60, 64), (1, 64, 4), (1, 0, 64)):
        assert b(256, batch, rows, cols, 256, 256, None, None, None) == BAD
    assert b(256, 65536, 64, 64, 256, 256, None, None, None) == UNSUPPORTED
    assert b(256, 1, 64, 64, None, None, None, None, None) == BAD


def test_routed_rows(mok):
    L, s = mok._lib, schedule(mok)
    p = ctypes.byref(s)
    for f in (L.mok_dispatch, L.mok_dispatch_backward, L.mok_combine):
        for width in (0, 4, 12, 16392, -8):
            assert f(p, 256, width, 256, None) == BAD
        assert f(p, None, 64, 256, None) == BAD and f(p, 256, 64, 264, None) == BAD and f(None, 256, 64, 256, None) == BAD
    assert L.mok_combine_backward(p, 256, 256, 64, 256, None, None) == BAD
    big = 1 << 24  # outputs over inputs: dispatch's rows and x, combine's rows and out, drows and rows but for the same buffer
    n = s.rpad_max * 128
    assert L.mok_dispatch(p, big + n - 16, 64, big, None) == BAD and L.mok_dispatch_backward(p, big, 64, big + 16, None) == BAD
    assert L.mok_combine(p, big, 64, big + n - 16, None) == BAD
    f = L.mok_combine_backward
    assert f(p, big, 2 * big, 64, big + 16, 3 * big, None) == BAD and f(p, big, 2 * big, 64, 2 * big, 3 * big, None) == BAD
    assert f(p, big, 2 * big, 64, 4 * big, big + 16, None) == BAD and f(p, big, 2 * big, 64, 4 * big, 256, None) == BAD
    assert L.mok_fp8_quantize_routed(p, 2, 256, 64, 256, 256, None, None, None) == BAD
    rows = s.rpad_max
    a, w = matrix(mok, rows=rows), matrix(mok, rows=16, batch=4, block=True)
    g = lambda a, w, out=256: L.mok_fp8_grouped_matmul(p, ctypes.byref(a), ctypes.byref(w), out, None)  # noqa: E731
    assert g(matrix(mok, rows=rows - 1), w) == BAD and g(a, matrix(mok, rows=16, batch=3, block=True)) == BAD
    assert g(a, matrix(mok, rows=12, batch=4, block=True)) == BAD and g(a, matrix(mok, rows=16, batch=4)) == BAD
    assert g(a, w, None) == BAD and g(a, matrix(mok, rows=16, cols=48, batch=4, block=True)) == BAD
    t = matrix(mok, rows=24, cols=rows, ld=(rows + 15) // 16 * 16)
    h = lambda a, b, out=256, dt=1: L.mok_fp8_grouped_wgrad(p, ctypes.byref(a), ctypes.byref(b), out, dt, None)  # noqa: E731
    assert h(a, t) == BAD and h(t, a) == BAD and h(t, t, None) == BAD and h(t, t, dt=3) == BAD
    huge = matrix(mok, rows=2**30, cols=rows, ld=t.ld)
    assert h(huge, t) == UNSUPPORTED  # rows of all experts' outputs beyond 31 bits
    for field, value in (("row_token", None), ("inv", None), ("meta", None), ("rpad_max", rows + 1), ("mblocks_max", 1)):
        bad = schedule(mok)
        setattr(bad, field, value)
        assert L.mok_dispatch(ctypes.byref(bad), 256, 64, 256, None) == BAD
        assert L.mok_fp8_grouped_matmul(ctypes.byref(bad), ctypes.byref(a), ctypes.byref(w), 256, None) == BAD
    s.topk_weights = None  # as under expert parallelism
    assert L.mok_combine(p, 256, 64, 256, None) == BAD
    empty = schedule(mok, T=0)
    assert L.mok_dispatch(ctypes.byref(empty), None, 64, None, None) == OK


def test_routes_workspace(mok):
    cfg, shape = mok.make_config(0, 0), mok.make_shape(8192, 128, 128, 128, 8)
    n = mok.mok_routes_workspace_bytes(cfg, shape)
    rows = 8192 * 8 + 128 * 127
    assert 4 * (3 * rows + 8192 * 8) <= n < mok.mok_workspace_bytes(cfg, shape) // 10
    with pytest.raises(mok.MokError):
        mok.mok_routes_workspace_bytes(cfg, mok.make_shape(16, 128, 128, 2, 3))
    s = mok.mok_schedule()
    f = lambda ws, n, ids=256: mok._lib.mok_build_routes(ctypes.byref(cfg), ctypes.byref(shape), ids, 256, ws, n,  # noqa: E731
                                                         ctypes.byref(s), None)
    assert f(None, n) == BAD and f(264, n) == BAD and f(256, n, None) == BAD and f(256, n - 1) == SMALL


def test_scales_weights_and_workspaces_over_inputs(mok):
    L, big = mok._lib, 1 << 24
    q = L.mok_fp8_quantize
    assert q(big, 4, 64, 2 * big, big + 496, None, None, None) == BAD  # scales over x
    assert q(big, 4, 64, None, None, 2 * big, big - 240, None) == BAD
    s = schedule(mok)
    p, n = ctypes.byref(s), s.rpad_max * 128
    assert L.mok_fp8_quantize_routed(p, 0, big, 64, 2 * big, big + n - 16, None, None, None) == BAD
    assert L.mok_fp8_quantize_blocks(big, 2, 64, 64, 2 * big, big + 16, None, None, None) == BAD
    assert L.mok_fp8_quantize_blocks(big, 2, 64, 64, None, None, 2 * big, big + 2 * 8192 - 16, None) == BAD
    s.topk_weights = big  # of combine: its output, and its gradient's
    assert L.mok_combine(p, 2 * big, 64, big, None) == BAD
    assert L.mok_combine_backward(p, 2 * big, 3 * big, 64, big, 4 * big, None) == BAD
    w = matrix(mok, block=True, q=1 << 22, s=1 << 23)
    f = lambda x, out, ws: L.mok_fp8_linear(x, 100, ctypes.byref(w), out, ws, 1 << 20, None, None)  # noqa: E731
    assert f(big, 2 * big, 2 * big) == BAD and f(big, 2 * big, 1 << 22) == BAD  # the workspace over out and w
    assert f(big, 2 * big, big) == BAD and f(big, 2 * big, (1 << 23) - 256) == BAD  # over x; over w's scales


# ---- the binding ----
def placed(mok, device="cuda:0", T=4, E=2, K=1):
    ws = _tensors(device, ws=(64, U8))["ws"]
    return mok.Schedule(schedule(mok, T, E, K), ws, None, None)


def calls(mok, at, where=None):
    """{call: (function, arguments)} on cuda:0, with the tensor named `where` on `at`."""
    R = 4 + 2 * 127
    shapes = dict(x=(4, 64, BF), rows=(R, 64, BF), dout=(4, 64, BF), out=(4, 16, BF), w=(16, 64, BF), status=(1, I32), drows=(R, 64, BF),
                  grows=(R, 16, BF), dw=(2, 16, 16, F32))
    shapes.update({"a.q": (4, 64, U8), "a.s": (1, 4, F32), "b.q": (16, 64, U8), "b.s": (1, 1, F32), "r.q": (R, 64, U8),
                   "r.s": (1, 260, F32), "e.q": (2, 16, 64, U8), "e.s": (2, 1, 1, F32), "t.q": (16, 272, U8), "t.s": (3, 16, F32),
                   "u.q": (16, 272, U8), "u.s": (3, 16, F32)})
    t = {k: _tensors(at if k == where else "cuda:0", **{k: v})[k] for k, v in shapes.items()}
    m = lambda k, cols, block=False: mok.Fp8(t[k + ".q"], t[k + ".s"], cols, block)  # noqa: E731
    s = placed(mok, at if where == "schedule" else "cuda:0")
    return {
        "dispatch": (mok.dispatch, (s, t["x"], t["rows"])),
        "dispatch_backward": (mok.dispatch_backward, (s, t["rows"], t["dout"])),
        "combine": (mok.combine, (s, t["rows"], t["dout"])),
        "combine_backward": (mok.combine_backward, (s, t["rows"], t["dout"], t["drows"])),
        "fp8_matmul": (mok.fp8_matmul, (m("a", 64), m("b", 64, True), BF, t["out"], t["status"])),
        "fp8_linear": (mok.fp8_linear, (t["x"], m("b", 64, True), t["out"], t["status"])),
        "quantize routed": (mok.fp8_quantize, (t["rows"], False, True, s)),
        "dispatch_fp8": (mok.dispatch_fp8, (s, t["x"])),
        "fp8_grouped_matmul": (mok.fp8_grouped_matmul, (s, m("r", 64), m("e", 64, True), t["grows"])),
        "fp8_grouped_wgrad": (mok.fp8_grouped_wgrad, (s, m("t", R), m("u", R), F32, t["dw"])),
    }


AWAY = [("dispatch", "x"), ("dispatch", "rows"), ("dispatch", "schedule"), ("dispatch_backward", "rows"), ("dispatch_backward", "dout"),
        ("combine", "rows"), ("combine", "dout"), ("combine_backward", "dout"), ("combine_backward", "drows"),
        ("combine_backward", "schedule"), ("fp8_matmul", "a.s"), ("fp8_matmul", "b.q"), ("fp8_matmul", "b.s"), ("fp8_matmul", "out"),
        ("fp8_matmul", "status"), ("fp8_linear", "b.q"), ("fp8_linear", "b.s"), ("fp8_linear", "out"), ("fp8_linear", "status"),
        ("quantize routed", "rows"), ("quantize routed", "schedule"), ("dispatch_fp8", "x"), ("fp8_grouped_matmul", "r.q"),
        ("fp8_grouped_matmul", "r.s"), ("fp8_grouped_matmul", "e.q"), ("fp8_grouped_matmul", "e.s"), ("fp8_grouped_matmul", "grows"),
        ("fp8_grouped_matmul", "schedule"), ("fp8_grouped_wgrad", "t.s"), ("fp8_grouped_wgrad", "u.q"), ("fp8_grouped_wgrad", "dw"),
        ("fp8_grouped_wgrad", "schedule")]


@pytest.mark.parametrize("call,where", AWAY)
def test_operands_on_another_device_are_refused(mok, call, where):
    f, args = calls(mok, "cuda:1", where)[call]
    with pytest.raises(ValueError, match="must be on cuda:[01].*got cuda:[01]"):
        f(*args)


@pytest.mark.parametrize("call", ["dispatch", "combine", "combine_backward", "fp8_matmul", "fp8_linear", "dispatch_fp8",
                                  "fp8_grouped_matmul", "fp8_grouped_wgrad", "quantize routed"])
def test_streams_of_another_device_are_refused(mok, monkeypatch, call):
    streams = _Streams(monkeypatch)
    f, args = calls(mok, "cuda:0")[call]
    with pytest.raises(ValueError, match="stream must be on cuda:0.*got cuda:1"):
        f(*args, stream=streams.Stream(0x5550, 1))


@pytest.mark.parametrize("call", ["dispatch", "dispatch_backward", "combine", "combine_backward", "fp8_matmul", "fp8_linear",
                                  "dispatch_fp8", "fp8_grouped_matmul", "fp8_grouped_wgrad"])
def test_a_given_stream_is_current_for_the_call(mok, monkeypatch, call):
    """What a call allocates belongs to the stream that it was given."""
    streams = _Streams(monkeypatch)
    f, args = calls(mok, "cuda:0")[call]
    at = []

    class Bind:
        def __getattr__(self, name):
            return lambda *a: at.append([s.cuda_stream for s in streams.current]) or (None, None, None, None)
    monkeypatch.setattr(mok, "_bind", Bind())
    f(*args, stream=0x5550)
    assert at == [[0x5550]] and not streams.current


def test_what_is_no_8bit_matrix_is_named(mok):
    q, s = torch.zeros((4, 64), dtype=U8), torch.zeros((1, 4))
    a = mok.Fp8(q, s, 64)
    for bad, name in ((None, "b must"), (q, "b must"), (mok.Fp8(q.float(), s, 64), "b.q"),
                      (mok.Fp8(q[:, :40], s, 40), "b.q's rows"), (mok.Fp8(q, s, 65), "b.q's rows"), (mok.Fp8(q[None], s, 64), "b.q must"),
                      (mok.Fp8(q, None, 64), "b.s must")):
        with pytest.raises(ValueError, match=name):
            mok.fp8_matmul(a, bad)
    t = _tensors("cuda:0", q=(4, 64, U8), s=(1, 4, F32), short=(1, 3, F32))
    c = mok.Fp8(t["q"], t["s"], 64)
    for bad in (mok.Fp8(t["q"], t["short"], 64), mok.Fp8(t["q"], t["s"], 64, True)):
        with pytest.raises(ValueError, match="b.s must have shape"):
            mok.fp8_matmul(c, bad)
    with pytest.raises(ValueError, match="a.q must be a CUDA tensor"):
        mok.fp8_matmul(a, mok.Fp8(q, torch.zeros((1, 1)), 64, True))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        mok.fp8_quantize(torch.zeros((4, 64), dtype=BF))
    with pytest.raises(ValueError, match="w must be a CUDA tensor"):
        mok.fp8_quantize_weight(torch.zeros((8, 64), dtype=BF))
    assert a.rows == 4
