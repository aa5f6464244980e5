"""Routed rows as calls of their own, on the GPU vs tests/fp8_ref.py.

dispatch moves bf16 values: equal bits.  Sums are fp32 fused multiply-adds in ascending order, K of them: off by K 2^-24 of
the sum of the magnitudes, and rounded to bf16 (half a step, 2^-8 of the value); drows is one fp32 product rounded to
bf16: 2^-24 more; a weight's gradient adds up W products in fp32, in any order: W 2^-24 of the magnitudes."""
import ctypes

import pytest
import torch

import fp8_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 2.0**-24


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return g, lambda *s: torch.randn(s, generator=g, device="cuda")


def routing(kind, T, E, K, seed=0):
    g, _ = gen(seed)
    if kind == "one":           # all slots on the last expert: the same index K times for a token
        ids = torch.full((T, K), E - 1, device="cuda")
    elif kind == "few":         # most experts without a row
        ids = torch.randint(0, min(E, 2), (T, K), generator=g, device="cuda")
    elif kind == "invalid":     # ids outside the experts among them, whole tokens without one
        ids = torch.randint(-2, E + 3, (T, K), generator=g, device="cuda")
        ids[: T // 3] = -1
    else:
        ids = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices
    w = torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    return ids.to(torch.int32), w


CASES = [(1, 8, 3, 64, "spread"), (1, 128, 8, 4096, "spread"), (3, 4, 4, 8, "spread"), (130, 5, 2, 136, "one"), (257, 16, 3, 1000, "few"),
         (300, 7, 2, 2056, "invalid"), (128, 1, 1, 256, "one"), (1003, 60, 5, 520, "spread"), (40, 1024, 32, 16, "spread"),
         (64, 300, 9, 7168, "spread"), (17, 12, 6, 16384, "invalid")]


def filled(rows, W, mok):
    return torch.full((rows, W), 7.0, dtype=BF, device="cuda")


@pytest.mark.parametrize("T,E,K,W,kind", CASES)
def test_rows_there_and_back(mok, T, E, K, W, kind):
    ids, w = routing(kind, T, E, K)
    routes = mok.Routes(T, E, K)
    sched = routes.build(ids, w)
    row, _, end = ref.layout(ids, E)
    R = routes.rows
    assert R == sched.c.rpad_max
    _, n = gen(T + W)
    x, y, dout = n(T, W).to(BF), n(R, W).to(BF), n(T, W).to(BF)
    out = filled(R, W, mok)
    assert mok.dispatch(sched, x, out=out) is not None
    assert torch.equal(out[:end], ref.dispatch(x, row, R)[:end])
    assert (out[end:] == 7).all()  # behind the layout's end: as it was
    for got, (want, mag) in ((mok.dispatch_backward(sched, y), ref.combine(y, row)), (mok.combine(sched, y), ref.combine(y, row, w))):
        assert ((got.to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * EPS * mag).all()
    drows, dw, mag = ref.combine_grads(y, dout, row, w)
    got = filled(R, W, mok)
    _, gw = mok.combine_backward(sched, y, dout, drows=got)
    assert ((got[:end].to(F64) - drows[:end]).abs() <= (2.0**-8 + EPS) * drows[:end].abs()).all()
    assert (got[end:] == 7).all()
    assert ((gw.to(F64) - dw).abs() <= (W + 1) * EPS * mag).all()
    same, gw2 = mok.combine_backward(sched, y, dout, drows=y)  # in the rows' own buffer
    assert same.data_ptr() == y.data_ptr() and torch.equal(y[:end], got[:end]) and torch.equal(gw2, gw)
    want_status = 1 << mok.MOK_ERR_BAD_EXPERT_ID if kind == "invalid" else 0
    assert mok.mok_read_device_status(sched) == want_status


def test_values_outside_the_layout_do_not_count(mok):
    """NaN in padding rows and behind the layout: sums and gradients do not see them; infinities in a token's own rows do."""
    T, E, K, W = 50, 6, 2, 72
    ids, w = routing("spread", T, E, K)
    sched = mok.Routes(T, E, K).build(ids, w)
    row, _, end = ref.layout(ids, E)
    y = torch.full((sched.c.rpad_max, W), float("nan"), dtype=BF, device="cuda")
    y[row.flatten().cuda()] = 1.0
    assert torch.isfinite(mok.combine(sched, y)).all() and (mok.dispatch_backward(sched, y) == K).all()
    dr, dw = mok.combine_backward(sched, y, torch.ones((T, W), dtype=BF, device="cuda"))
    assert torch.isfinite(dr[:end]).all() and (dw == W).all()
    y[row[7, 1], 3] = float("-inf")
    assert mok.combine(sched, y)[7, 3] == float("-inf")
    assert mok.combine_backward(sched, y, torch.ones((T, W), dtype=BF, device="cuda"))[1][7, 1] == float("-inf")


def test_no_tokens(mok):
    sched = mok.Routes(0, 4, 2).build(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), torch.zeros((0, 2), device="cuda"))
    x = torch.zeros((0, 64), dtype=BF, device="cuda")
    rows = filled(sched.c.rpad_max, 64, mok)
    assert (mok.dispatch(sched, x, out=rows) == 7).all()
    assert mok.combine(sched, rows).shape == (0, 64) and mok.dispatch_backward(sched, rows).shape == (0, 64)
    dr, dw = mok.combine_backward(sched, rows, x, drows=rows)
    assert (dr == 7).all() and dw.shape == (0, 2)


def test_on_the_layers_schedule(mok):
    """A schedule of mok_build_schedule and of mok_build_schedule_noalloc's kind (no workspace) serves as well."""
    T, E, K, H = 200, 8, 2, 256
    ids, w = routing("spread", T, E, K)
    cfg, shape = mok.make_config(128, 256), mok.make_shape(T, H, 128, E, K)
    full = mok.mok_build_schedule(cfg, shape, ids, w, mok.alloc_workspace(cfg, shape))
    lean = mok.Routes(T, E, K).build(ids, w)
    a, b = full.tables(), lean.tables()
    end = int(a["poff"][E])
    for k in ("counts", "offsets", "poff", "inv"):
        assert torch.equal(a[k], b[k]), k
    for k in ("perm", "row_token", "row_weight"):
        assert torch.equal(a[k][:end], b[k][:end]), k
    _, n = gen(1)
    x = n(T, H).to(BF)
    assert torch.equal(mok.dispatch(full, x)[:end], mok.dispatch(lean, x)[:end])
    with pytest.raises(mok.MokError):  # no staging for the layer
        mok.mok_forward(lean, x, mok.mok_weights(), x, torch.empty(1 << 24, dtype=torch.uint8, device="cuda"))


def test_refusals(mok):
    T, E, K, W = 16, 4, 2, 64
    ids, w = routing("spread", T, E, K)
    routes = mok.Routes(T, E, K)
    sched = routes.build(ids, w)
    x, rows = torch.zeros((T, W), dtype=BF, device="cuda"), torch.zeros((routes.rows, W), dtype=BF, device="cuda")
    bad = [(mok.dispatch, (sched, x[:-1]), "x"), (mok.dispatch, (sched, x.float()), "x"), (mok.dispatch, (sched, x, rows[:-1]), "out"),
           (mok.dispatch, (sched, x.cpu()), "x"), (mok.dispatch, (sched, None), "x"), (mok.dispatch, (sched, x.T), "x"),
           (mok.dispatch_backward, (sched, x), "drows"), (mok.combine, (sched, rows[:, ::2]), "rows"),
           (mok.combine, (sched, rows, x.float()), "out"), (mok.combine_backward, (sched, rows, rows), "dout"),
           (mok.combine_backward, (sched, rows, x, x), "drows"), (routes.build, (ids.long(), w), "topk_ids"),
           (routes.build, (ids, w[:-1]), "topk_weights"), (routes.build, (ids.cpu(), w), "topk_ids")]
    for call, args, name in bad:
        with pytest.raises(ValueError, match=name):
            call(*args)
    for width in (4, 12, 16392):
        with pytest.raises(mok.MokError):
            mok.dispatch(sched, torch.zeros((T, width), dtype=BF, device="cuda"))
    odd = torch.zeros(T * W + 1, dtype=BF, device="cuda")[1:].view(T, W)  # not on a 16-byte boundary
    with pytest.raises(mok.MokError):
        mok.dispatch(sched, odd)
    s = mok.mok_schedule.from_buffer_copy(sched.c)
    s.row_token = None
    for f in ("mok_dispatch", "mok_dispatch_backward", "mok_combine"):
        assert getattr(mok._lib, f)(ctypes.byref(s), x.data_ptr(), W, rows.data_ptr(), None) == mok.MOK_ERR_INVALID_ARG
    s = mok.mok_schedule.from_buffer_copy(sched.c)
    s.topk_weights = None  # as under expert parallelism
    assert mok._lib.mok_combine(ctypes.byref(s), rows.data_ptr(), W, x.data_ptr(), None) == mok.MOK_ERR_INVALID_ARG


def test_captured_and_replayed_on_another_stream(mok):
    """A step of build, dispatch, combine and gradients captured once, replayed with other routings."""
    T, E, K, W = 90, 6, 2, 256
    ids, w = routing("spread", T, E, K)
    routes = mok.Routes(T, E, K)
    _, n = gen(3)
    x, dout = n(T, W).to(BF), n(T, W).to(BF)
    rows, out, dx = filled(routes.rows, W, mok), torch.empty_like(x), torch.empty_like(x)

    def step():
        s = routes.build(ids, w)
        mok.dispatch(s, x, out=rows)
        mok.combine(s, rows, out=out)
        dr, dw = mok.combine_backward(s, rows, dout)
        mok.dispatch_backward(s, dr, out=dx)
        return dr, dw
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dr, dw = step()
    for kind in ("few", "spread", "one"):
        i2, w2 = routing(kind, T, E, K, seed=9)
        ids.copy_(i2), w.copy_(w2), rows.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        row, _, end = ref.layout(i2, E)
        assert torch.equal(rows[:end], ref.dispatch(x, row, end)) and (rows[end:] == 7).all()
        want, mag = ref.combine(rows, row, w2)
        assert ((out.to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * EPS * mag).all()
        assert torch.equal(mok.combine(routes.build(ids, w), rows), out)
        _, want_w, mag = ref.combine_grads(rows, dout, row, w2)
        assert ((dw.to(F64) - want_w).abs() <= (W + 1) * EPS * mag).all()
