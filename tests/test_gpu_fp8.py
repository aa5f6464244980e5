"""8-bit quantisation and products with a scale per 128 values, on the GPU vs tests/fp8_ref.py.

Quantisation: codes and scales are equal to the reference's, bit for bit but for the sign of zero.  Products: of the codes
and scales as they are, so what differs is fp32 arithmetic: up to 127 additions of a block's exact products, the scales' product, and
one fused multiply-add per block, 2^-24 of the sum of the magnitudes each; and the output's rounding (half a step: 2^-8
of the value in bf16).  A clustered split adds up to 8 partials: 7 more."""
import ctypes

import pytest
import torch

import fp8_ref as ref
from test_gpu_route import gen, routing

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def near(got, want, mag, blocks, what=""):
    tol = (128 + blocks + 8) * 2.0**-24 * mag + (2.0**-8 if got.dtype is BF else 2.0**-24) * want.abs()
    err = (got.to(F64) - want).abs()
    assert torch.isfinite(got.float()).all(), what
    assert (err <= tol).all(), (what, float((err / tol.clamp(min=1e-300)).max()))


def wild(R, C, seed):
    """Values over a wide range of magnitudes, blocks of zeros and of tiny ones among them."""
    g, n = gen(seed)
    x = n(R, C)
    rows = torch.randint(-40, 40, (R, 1), generator=g, device="cuda")
    cols = torch.randint(-3, 3, (1, C), generator=g, device="cuda")
    x = torch.ldexp(x, rows + cols)
    x[R // 2: R // 2 + 2] = 0
    x[:, C // 3: C // 3 + 1] = 0
    if R > 5:
        x[5] *= 1e-30  # below 2^-50
    return x.to(BF)


def same(codes, want):
    got = ref.decode(codes)
    off = torch.nonzero((got != want) & ~(torch.isnan(got) & torch.isnan(want)))
    assert len(off) == 0, (len(off), off[:4].tolist(), [(float(got[tuple(i)]), float(want[tuple(i)])) for i in off[:4]])


def same_scales(got, want):
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got).to(F64), torch.nan_to_num(want))


SHAPES = [(1, 8), (1, 128), (2, 136), (7, 1000), (127, 120), (128, 128), (129, 264), (300, 2056), (1003, 128)]


@pytest.mark.parametrize("R,C", SHAPES)
def test_quantize(mok, R, C):
    x = wild(R, C, R + C)
    if R > 8:
        x[3, C - 1], x[8, 0] = float("nan"), float("-inf")
    a, at = mok.fp8_quantize(x, transposed=True)
    q, s = ref.quantize(x, (1, 128))
    same(a.q[:, :C].contiguous(), q)
    same_scales(a.s[:, :R].T, s)
    assert (a.q[:, C:] == 0).all()
    qt, st = ref.quantize(x, (128, 1))
    same(at.q[:, :R].contiguous(), qt.T)
    same_scales(at.s[:, :C], st)
    assert (at.q[:, R:] == 0).all()
    only, none = mok.fp8_quantize(x)
    assert none is None and torch.equal(only.q, a.q) and torch.equal(only.s[:, :R].nan_to_num(), a.s[:, :R].nan_to_num())
    none, only = mok.fp8_quantize(x, rows=False, transposed=True)
    assert none is None and torch.equal(only.q, at.q)


@pytest.mark.parametrize("shape", [(8, 8), (128, 256), (136, 120), (1000, 2056), (3, 136, 264), (5, 8, 128)])
def test_quantize_weight(mok, shape):
    x = torch.stack([wild(*shape[-2:], 7 + e) for e in range(shape[0])]) if len(shape) == 3 else wild(*shape, 7)
    if x.shape[-2] > 8:
        x[..., 3, 5] = float("inf")
    N, K = shape[-2:]
    w, wt = mok.fp8_quantize_weight(x, transposed=True)
    for e in range(shape[0]) if len(shape) == 3 else (None,):
        xe, qe, se, qte, ste = ((x, w.q, w.s, wt.q, wt.s) if e is None else (x[e], w.q[e], w.s[e], wt.q[e], wt.s[e]))
        q, s = ref.quantize(xe, (128, 128))
        same(qe[:, :K].contiguous(), q)
        same_scales(se, s)
        same(qte[:, :N].contiguous(), q.T)
        same_scales(ste, s.T)
        assert (qe[:, K:] == 0).all() and (qte[:, N:] == 0).all()


def codes(R, C, seed, block=False, batch=None, mok=None):
    """An Fp8 of random codes (no NaN) and scales, as a checkpoint has them."""
    g, n = gen(seed)
    ld = (C + 15) // 16 * 16
    lead = () if batch is None else (batch,)
    q = n(*lead, R, ld).mul(30).to(torch.float8_e4m3fn)
    shape = (-(-R // 128), -(-C // 128)) if block else (-(-C // 128), (R + 3) // 4 * 4)
    s = torch.exp(n(*lead, *shape))
    return mok.Fp8(q, s, C, block)


def both(a, b):
    """(a b^T, sum of the magnitudes) of 64-bit matrices."""
    return a @ b.T, a.abs() @ b.abs().T


PRODUCTS = [(1, 8, 8), (1, 128, 128), (1, 2048, 7168), (2, 136, 264), (8, 64, 1024), (16, 1000, 392), (17, 264, 2056), (33, 128, 4096),
            (61, 7168, 2048), (64, 8, 520), (65, 392, 1032), (100, 136, 128), (128, 256, 1024), (129, 264, 520), (255, 1000, 136),
            (257, 1032, 2056), (600, 520, 1000), (1003, 1000, 2056), (1200, 2056, 264)]


@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_matmul(mok, M, N, K, block):
    a, b = codes(M, K, M + N, mok=mok), codes(N, K, K, block=block, mok=mok)
    want, mag = both(ref.of(a), ref.of(b))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for dt in (F32, BF):
        near(mok.fp8_matmul(a, b, out_dtype=dt, status=status), want, mag, -(-K // 128), dt)
    assert int(status) == 0


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear(mok, M, N, K):
    _, n = gen(M)
    x, w = n(M, K).to(BF), codes(N, K, 1, block=True, mok=mok)
    y = mok.fp8_linear(x, w)
    a, _ = mok.fp8_quantize(x)
    want, mag = both(ref.of(a), ref.of(w))
    near(y, want, mag, -(-K // 128))
    near(mok.fp8_matmul(a, w), want, mag, -(-K // 128))
    assert torch.equal(y, mok.fp8_linear(x, w, out=torch.empty_like(y)))  # from run to run


def test_linear_gradients(mok):
    """Both gradients against the formulas on the operands as they were quantised."""
    M, N, K = 300, 264, 520
    _, n = gen(5)
    x, dy, w = n(M, K).to(BF), n(M, N).to(BF), (n(N, K) * 0.02).to(BF)
    wq, wt = mok.fp8_quantize_weight(w, transposed=True)
    (d, dt), (_, xt) = mok.fp8_quantize(dy, transposed=True), mok.fp8_quantize(x, transposed=True, rows=False)
    assert torch.equal(ref.of(wt), ref.of(wq).T)
    near(mok.fp8_matmul(d, wt), *both(ref.of(d), ref.of(wt)), 3)
    dw = mok.fp8_matmul(dt, xt, out_dtype=F32)
    near(dw, *both(ref.of(dt), ref.of(xt)), 3)
    # and of the function itself, to the operands' rounding: each is off by 2^-4 of its value at most, or by half the
    # smallest step, 2^-10 of a scale of at most amax / 448
    tol = lambda v: v.abs() * 2.0**-4 + v.abs().amax() * 2.0**-18  # noqa: E731
    x64, dy64 = x.to(F64), dy.to(F64)
    bound = (dy64.abs() + tol(dy64)).T @ (x64.abs() + tol(x64)) - dy64.abs().T @ x64.abs()
    assert ((dw.to(F64) - dy64.T @ x64).abs() <= bound * (1 + 1e-3)).all()


def test_special_values(mok):
    """NaN and infinity in a row make that row NaN and no other; an infinite scale product is the documented limit."""
    M, N, K = 40, 136, 264
    _, n = gen(6)
    x, w = n(M, K).to(BF), codes(N, K, 1, block=True, mok=mok)
    clean = mok.fp8_linear(x, w)
    x[3, 200], x[17, 0] = float("nan"), float("inf")
    y = mok.fp8_linear(x, w)
    assert torch.isnan(y[[3, 17]]).all()
    keep = [i for i in range(M) if i not in (3, 17)]
    assert torch.equal(y[keep], clean[keep])
    assert (mok.fp8_linear(torch.zeros_like(x), w) == 0).all()


GROUPED = [(1, 8, 3, 64, 72, "spread"), (1, 128, 8, 4096, 1536, "spread"), (2, 4, 4, 8, 8, "one"), (130, 5, 2, 136, 264, "one"),
           (257, 16, 3, 1000, 136, "few"), (300, 7, 2, 520, 128, "invalid"), (90, 40, 5, 264, 1032, "spread"), (512, 2, 2, 128, 256, "spread"),
           (1003, 12, 3, 2056, 520, "spread"), (40, 1024, 32, 128, 64, "spread"), (2000, 3, 2, 392, 2056, "few")]


@pytest.mark.parametrize("T,E,K,H,N,kind", GROUPED)
def test_grouped(mok, T, E, K, H, N, kind):
    """Dispatch in 8 bits, the product, both gradients, on routings that leave experts empty and tokens without a row."""
    ids, w = routing(kind, T, E, K)
    sched = mok.Routes(T, E, K).build(ids, w)
    row, segments, end = ref.layout(ids, E)
    R = sched.c.rpad_max
    _, n = gen(T + N)
    x = n(T, H).to(BF)
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    live[row[row >= 0].cuda()] = True
    xr = ref.dispatch(x, row, R)
    a, at = mok.dispatch_fp8(sched, x, transposed=True)
    plain, plain_t = mok.fp8_quantize(xr, transposed=True)
    assert torch.equal(a.q[live], plain.q[live]) and torch.equal(a.s[:, :R][:, live], plain.s[:, :R][:, live])
    assert torch.equal(at.q[:, :end], plain_t.q[:, :end]) and torch.equal(at.s[: end // 128], plain_t.s[: end // 128])
    # routed rows with anything in the padding
    junk = torch.where(live[:, None], xr, torch.full_like(xr, float("nan")))
    b, bt = mok.fp8_quantize(junk, transposed=True, sched=sched)
    assert torch.equal(b.q[live], a.q[live]) and torch.equal(bt.q[:, :end], at.q[:, :end])
    only, _ = mok.dispatch_fp8(sched, x)
    assert torch.equal(only.q[live], a.q[live]) and torch.equal(only.s[:, :R][:, live], a.s[:, :R][:, live])
    weights = codes(N, H, 3, block=True, batch=E, mok=mok)
    out = torch.full((R, N), 7.0, dtype=BF, device="cuda")
    y = mok.fp8_grouped_matmul(sched, only, weights, out=out)
    assert (out[~live] == 7).all()  # padding, and what lies behind the layout
    dyr = torch.where(live[:, None], n(R, N), torch.zeros((), device="cuda")).to(BF)
    d, dt = mok.fp8_quantize(dyr, transposed=True, sched=sched)
    dws = {dt_: mok.fp8_grouped_wgrad(sched, dt, at, out_dtype=dt_) for dt_ in (F32, BF)}
    ax, ad, adt = (ref.values(ref.decode(m.q)[:, :m.cols], m.s[:, :m.rows].T, (1, 128)) for m in (plain, d, dt))
    axt = ref.values(ref.decode(plain_t.q)[:, :R], plain_t.s[:, :H].T, (1, 128))
    for e, (r0, rn) in enumerate(segments):
        if rn:
            near(y[r0:r0 + rn], *both(ax[r0:r0 + rn], ref.of(weights, e)), -(-H // 128), ("y", e))
        for dw in dws.values():
            if rn:
                near(dw[e], *both(adt[:, r0:r0 + rn], axt[:, r0:r0 + rn]), -(-rn // 128), ("dw", e))
            else:
                assert (dw[e] == 0).all()
    del ad
    assert mok.mok_read_device_status(sched) in (0, 1 << mok.MOK_ERR_BAD_EXPERT_ID)


def test_expert_block_of_these_calls(mok):
    """A gated block per expert from the calls, as a user runs them: dispatch, gate and up, activation, down, combine."""
    T, E, K, H, I = 200, 6, 2, 384, 264
    ids, wts = routing("spread", T, E, K)
    sched = mok.Routes(T, E, K).build(ids, wts)
    row, segments, end = ref.layout(ids, E)
    _, n = gen(8)
    x = n(T, H).to(BF)
    wg, wu, wd = ((n(E, *s) * 0.05).to(BF) for s in ((I, H), (I, H), (H, I)))
    qg, qu, qd = (mok.fp8_quantize_weight(m)[0] for m in (wg, wu, wd))
    a, _ = mok.dispatch_fp8(sched, x)
    R = sched.c.rpad_max
    buf = lambda w: torch.zeros((R, w), dtype=BF, device="cuda")  # noqa: E731
    g, u = mok.fp8_grouped_matmul(sched, a, qg, out=buf(I)), mok.fp8_grouped_matmul(sched, a, qu, out=buf(I))
    act = (torch.nn.functional.silu(g.float()) * u.float()).to(BF)
    b, _ = mok.fp8_quantize(act, sched=sched)
    y = mok.fp8_grouped_matmul(sched, b, qd, out=buf(H))
    out = mok.combine(sched, y)
    # the reference takes each stage's own input, so that no rounding counts twice
    xq = ref.values(*ref.quantize(x, (1, 128)), (1, 128))
    bq = ref.values(*ref.quantize(act, (1, 128)), (1, 128))
    for e, (r0, rn) in enumerate(segments):
        if rn:
            t = torch.nonzero((row >= r0) & (row < r0 + rn))[:, 0].cuda()
            order = row[row >= 0][(row[row >= 0] >= r0) & (row[row >= 0] < r0 + rn)].argsort().cuda()
            near(g[r0:r0 + rn], *both(xq[t[order]], ref.of(qg, e)), 3, "g")
            near(u[r0:r0 + rn], *both(xq[t[order]], ref.of(qu, e)), 3, "u")
            near(y[r0:r0 + rn], *both(bq[r0:r0 + rn], ref.of(qd, e)), 3, "y")
    want, mag = ref.combine(y, row, wts)
    assert ((out.to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * 2.0**-24 * mag).all()


def test_captured_and_replayed(mok):
    """Two graphs of the same call at work at once, and a replay with other inputs."""
    M, N, K = 48, 264, 1032
    _, n = gen(9)
    w = codes(N, K, 1, block=True, mok=mok)
    xs = [n(M, K).to(BF) for _ in range(2)]
    mok.fp8_linear(xs[0], w)
    torch.cuda.synchronize()
    graphs, ys = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys.append(mok.fp8_linear(x, w))
        graphs.append(g)
    for k in range(3):
        for x in xs:
            x.copy_(n(M, K))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, y in zip(xs, ys):
            assert torch.equal(y, mok.fp8_linear(x, w))


def test_nothing_to_sum_and_no_rows(mok):
    a = mok.Fp8(torch.zeros((5, 0), dtype=torch.uint8, device="cuda"), torch.zeros((0, 8), device="cuda"), 0)
    b = mok.Fp8(torch.zeros((16, 0), dtype=torch.uint8, device="cuda"), torch.zeros((0, 16), device="cuda"), 0)
    assert (mok.fp8_matmul(a, b) == 0).all() and (mok.fp8_matmul(a, b, out_dtype=F32) == 0).all()
    w = codes(16, 64, 1, block=True, mok=mok)
    assert mok.fp8_linear(torch.zeros((0, 64), dtype=BF, device="cuda"), w).shape == (0, 16)
    q, qt = mok.fp8_quantize(torch.zeros((0, 64), dtype=BF, device="cuda"), transposed=True)
    assert q.q.shape == (0, 64) and qt.q.shape == (64, 0)
    sched = mok.Routes(0, 4, 2).build(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), torch.zeros((0, 2), device="cuda"))
    x, xt = mok.dispatch_fp8(sched, torch.zeros((0, 64), dtype=BF, device="cuda"), transposed=True)
    mok.fp8_grouped_matmul(sched, x, codes(16, 64, 1, block=True, batch=4, mok=mok))
    assert (mok.fp8_grouped_wgrad(sched, xt, xt) == 0).all()


def test_refusals(mok):
    a, b, w = codes(32, 64, 1, mok=mok), codes(16, 64, 2, mok=mok), codes(16, 64, 3, block=True, mok=mok)
    x = torch.zeros((32, 64), dtype=BF, device="cuda")
    ids, wt = routing("spread", 16, 4, 2)
    sched = mok.Routes(16, 4, 2).build(ids, wt)
    R = sched.c.rpad_max
    ra, we = codes(R, 64, 1, mok=mok), codes(16, 64, 2, block=True, batch=4, mok=mok)
    ta, tb = codes(24, R, 1, mok=mok), codes(16, R, 2, mok=mok)
    F = mok.Fp8
    bad = [(mok.fp8_matmul, (F(a.q, a.s[:-1], 64), b), "a.s"), (mok.fp8_matmul, (F(a.q.float(), a.s, 64), b), "a.q"),
           (mok.fp8_matmul, (F(a.q, a.s, 65), b), "a.q"), (mok.fp8_matmul, (w, b), "a must"), (mok.fp8_matmul, (a, F(b.q, b.s, 48)), "a and b"),
           (mok.fp8_matmul, (a, b, torch.float16), "out_dtype"), (mok.fp8_matmul, (a, b, F32, x), "out"),
           (mok.fp8_matmul, (a, F(b.q.cpu(), b.s, 64)), "b.q"), (mok.fp8_matmul, (a, F(b.q, b.s.half(), 64)), "b.s"),
           (mok.fp8_matmul, (a, None), "b must"), (mok.fp8_linear, (x, a), "w must"),
           (mok.fp8_matmul, (a, b, F32, None, torch.zeros(2, dtype=torch.int32, device="cuda")), "status"),
           (mok.fp8_linear, (x, b), "w must"), (mok.fp8_linear, (x.float(), w), "x"), (mok.fp8_linear, (x[:, :32], w), "x"),
           (mok.fp8_linear, (x, w, x), "out"), (mok.fp8_linear, (None, w), "x"), (mok.fp8_quantize, (x.float(),), "x"),
           (mok.fp8_quantize, (x[:, ::2],), "x"), (mok.fp8_quantize, (x, False, True, sched), "x"), (mok.fp8_quantize_weight, (x.float(),), "w"),
           (mok.dispatch_fp8, (sched, x), "x"), (mok.fp8_grouped_matmul, (sched, a, we), "a.q"),
           (mok.fp8_grouped_matmul, (sched, ra, w), "w"), (mok.fp8_grouped_matmul, (sched, ra, F(we.q[:3], we.s[:3], 64, True)), "w.q"),
           (mok.fp8_grouped_matmul, (sched, ra, we, x), "out"), (mok.fp8_grouped_wgrad, (sched, a, tb), "a must"),
           (mok.fp8_grouped_wgrad, (sched, ta, w), "b must"), (mok.fp8_grouped_wgrad, (sched, ta, tb, BF, x), "out")]
    for call, args, name in bad:
        with pytest.raises(ValueError, match=name):
            call(*args)
    with pytest.raises(mok.MokError):
        mok.fp8_quantize(torch.zeros((4, 12), dtype=BF, device="cuda"))
    with pytest.raises(mok.MokError):
        mok.fp8_quantize(x, rows=False)  # nothing asked for
    with pytest.raises(mok.MokError):
        mok.fp8_quantize_weight(torch.zeros((12, 64), dtype=BF, device="cuda"))
    with pytest.raises(mok.MokError):  # an output of 12 columns
        mok.fp8_matmul(a, codes(12, 64, 1, mok=mok))
    odd = torch.zeros(32 * 64 + 16, dtype=torch.uint8, device="cuda")[8:8 + 32 * 64].view(32, 64)  # not on a 16-byte boundary
    with pytest.raises(mok.MokError):
        mok.fp8_matmul(F(odd, a.s, 64), b)
    m = mok.mok_fp8_matrix(a.q.data_ptr(), a.s.data_ptr(), 32, 64, 64, 1, mok.MOK_FP8_ROWS)
    p = ctypes.byref(m)
    out = torch.zeros((32, 32), dtype=F32, device="cuda")
    assert mok._lib.mok_fp8_matmul(p, p, out.data_ptr(), 5, None, None) == mok.MOK_ERR_INVALID_ARG
    m.ld = 40
    assert mok._lib.mok_fp8_matmul(p, p, out.data_ptr(), mok.MOK_DT_FP32, None, None) == mok.MOK_ERR_INVALID_ARG
    assert mok._lib.mok_fp8_linear_workspace_bytes(4, 12) == 0 and mok._lib.mok_fp8_linear_workspace_bytes(-1, 64) == 0
