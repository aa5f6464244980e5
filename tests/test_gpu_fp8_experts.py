"""The experts' data gradient, every quantiser on values of all magnitudes, and forms of the per-expert calls that the other
files leave out, on the GPU vs tests/fp8_ref.py (tests/test_gpu_fp8.py and tests/test_gpu_route.py have the tolerances)."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import both, near, same, same_scales, wild
from test_gpu_route import EPS, gen, routing

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def routed(mok, kind, T, E, K, seed=0):
    """(schedule, row of each slot, segments, the layout's end, rows that hold a slot)."""
    ids, w = routing(kind, T, E, K, seed)
    sched = mok.Routes(T, E, K).build(ids, w)
    row, segments, end = ref.layout(ids, E)
    live = torch.zeros(sched.c.rpad_max, dtype=torch.bool, device="cuda")
    live[row[row >= 0].cuda()] = True
    return sched, row, segments, end, live


@pytest.mark.parametrize("T,E,K,H,N,kind", [(1, 8, 3, 136, 264, "spread"), (130, 5, 2, 264, 136, "one"), (300, 7, 2, 520, 392, "invalid"),
                                            (257, 16, 3, 1000, 136, "few"), (700, 6, 2, 392, 1000, "spread"), (40, 12, 4, 128, 8, "spread")])
def test_data_gradient(mok, T, E, K, H, N, kind):
    """dx of y[r] = x[token of r] w[expert of r]^T: dy's rows times the transposed codes of real weights, summed over a token's
    rows.  Each stage against 64 bits on its own input, and the product against the formula without quantisation."""
    sched, row, segments, _, live = routed(mok, kind, T, E, K)
    _, n = gen(T + H)
    w = (n(E, N, H) * 0.05).to(BF)
    wq, wt = mok.fp8_quantize_weight(w, transposed=True)
    dy = torch.where(live[:, None], n(sched.c.rpad_max, N), torch.full((), float("nan"), device="cuda")).to(BF)
    d, _ = mok.fp8_quantize(dy, sched=sched)
    rows = mok.fp8_grouped_matmul(sched, d, wt, out=torch.zeros((sched.c.rpad_max, H), dtype=BF, device="cuda"))
    assert (rows[~live] == 0).all()
    dq = ref.values(ref.decode(d.q)[:, :N], d.s[:, :d.rows].T, (1, 128))
    # a rounding to E4M3: 2^-4 of the value, or half the smallest step, 2^-10 of a scale of at most amax / 448
    tol = lambda v: v.abs() * 2.0**-4 + v.abs().amax() * 2.0**-18  # noqa: E731
    for e, (r0, rn) in enumerate(segments):
        if not rn:
            continue
        we = ref.of(wt, e)
        assert torch.equal(we, ref.of(wq, e).T)
        want, mag = both(dq[r0:r0 + rn], we)
        near(rows[r0:r0 + rn], want, mag, -(-N // 128), e)
        d64, w64 = dy[r0:r0 + rn].to(F64), w[e].to(F64)
        off = (d64.abs() + tol(d64)) @ (w64.abs() + tol(w64)) - d64.abs() @ w64.abs()
        off = off + (128 + N // 128 + 9) * 2.0**-24 * mag + 2.0**-8 * want.abs()
        assert ((rows[r0:r0 + rn].to(F64) - d64 @ w64).abs() <= off * (1 + 1e-6)).all()
    want, mag = ref.combine(rows, row)
    assert ((mok.dispatch_backward(sched, rows).to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * EPS * mag).all()


def unit(N, mok):
    """The identity as a matrix with scales of 1 per 128 x 128 values."""
    q = torch.zeros((N, (N + 15) // 16 * 16), device="cuda")
    q[torch.arange(N), torch.arange(N)] = 1.0
    b = -(-N // 128)
    return mok.Fp8(q.to(torch.float8_e4m3fn), torch.ones((b, b), device="cuda"), N, True)


@pytest.mark.parametrize("C", [8, 120, 128, 136, 392, 1000])
@pytest.mark.parametrize("M", [1, 3, 8, 9])
def test_values_that_a_linear_quantises_itself(mok, M, C):
    """Times the identity, few rows (and one more, which are quantised by a kernel of their own) come back as their codes' values,
    rounded to fp32 and to bf16: bit for bit, over all magnitudes.  A NaN or an infinity in any block takes its row."""
    x = torch.cat([wild(64, C, M + C)[3:6], wild(64, C, M + C + 1)[30:36]])[:M]
    q, s = ref.quantize(x, (1, 128))
    y = mok.fp8_linear(x, unit(C, mok))
    assert torch.equal(y, ref.values(q, s, (1, 128)).to(F32).to(BF))
    bad = x.clone()
    bad[M - 1, C - 1] = float("nan") if M & 2 else float("-inf")
    got = mok.fp8_linear(bad, unit(C, mok))
    assert torch.isnan(got[M - 1]).all() and torch.equal(got[:M - 1], y[:M - 1])


@pytest.mark.parametrize("M", [1, 3, 8])
def test_special_values_in_few_rows(mok, M):
    """As for many rows: a NaN or an infinity, also in the last and partial K block, makes its own row NaN and no other."""
    N, K = 136, 1032
    g, n = gen(M)
    x = n(M, K).to(BF)
    w = mok.fp8_quantize_weight((n(N, K) * 0.05).to(BF))[0]
    clean = mok.fp8_linear(x, w)
    for value in (float("nan"), float("inf"), float("-inf")):
        for col in (0, 500, K - 8, K - 1):
            r = col % M
            bad = x.clone()
            bad[r, col] = value
            y = mok.fp8_linear(bad, w)
            keep = [i for i in range(M) if i != r]
            assert torch.isnan(y[r]).all() and torch.equal(y[keep], clean[keep])
    assert (mok.fp8_linear(torch.zeros_like(x), w) == 0).all()


@pytest.mark.parametrize("T,E,K,W,kind", [(1, 8, 3, 8, "spread"), (90, 5, 2, 136, "spread"), (200, 7, 2, 1000, "invalid"), (64, 64, 40, 1160, "spread"),
                                          (130, 3, 3, 2056, "one")])
def test_dispatch_of_all_magnitudes(mok, T, E, K, W, kind):
    """Codes on the dispatch gather, rows alone and both ways, equal the reference's on values of all magnitudes, with NaN and
    infinity among them; codes behind the columns are zeros; more than 32 slots of a token."""
    sched, row, _, end, live = routed(mok, kind, T, E, K)
    x = wild(T, W, T + W)
    if T > 8:
        x[2, W - 1], x[8, 0], x[7, W // 2] = float("nan"), float("-inf"), float("inf")
    rows = ref.dispatch(x, row, sched.c.rpad_max)
    q, s = ref.quantize(rows, (1, 128))
    only, _ = mok.dispatch_fp8(sched, x)
    a, at = mok.dispatch_fp8(sched, x, transposed=True)
    for m in (only, a):
        same(m.q[live][:, :W].contiguous(), q[live])
        same_scales(m.s[:, :m.rows][:, live].T, s[live])
        assert (m.q[live][:, W:] == 0).all()
    qt, st = ref.quantize(rows, (128, 1))
    qt = torch.where(live[:, None], qt, torch.zeros((), dtype=F64, device="cuda"))  # padding rows of a NaN's block are zeros all the same
    same(at.q[:, :end].contiguous(), qt[:end].T)
    same_scales(at.s[:end // 128, :W], st[:end // 128])


def test_as_many_experts_as_there_may_be(mok):
    """1024 experts with some 50 rows each: units that every CTA pair counts for itself, three experts per thread."""
    T, E, K, H, N = 6400, 1024, 8, 136, 72
    sched, _, segments, _, live = routed(mok, "spread", T, E, K)
    assert T * K >= 48 * E and min(rn for _, rn in segments) > 0
    _, n = gen(1)
    a, _ = mok.dispatch_fp8(sched, n(T, H).to(BF))
    w = mok.fp8_quantize_weight((n(E, N, H) * 0.05).to(BF))[0]
    y = mok.fp8_grouped_matmul(sched, a, w, out=torch.full((sched.c.rpad_max, N), 7.0, dtype=BF, device="cuda"))
    assert (y[~live] == 7).all()
    ax = ref.values(ref.decode(a.q)[:, :H], a.s[:, :a.rows].T, (1, 128))
    for e, (r0, rn) in enumerate(segments):
        near(y[r0:r0 + rn], *both(ax[r0:r0 + rn], ref.of(w, e)), 2, e)


@pytest.mark.parametrize("T,E", [(60, 12), (900, 6)])
def test_captured_experts_step(mok, T, E):
    """Routing, dispatch, product, both gradients in one graph, replayed with other routings and values: bits as in eager calls."""
    K, H, N = 2, 264, 392
    ids, wts = routing("spread", T, E, K)
    _, n = gen(T)
    x, dout, w = n(T, H).to(BF), n(T, N).to(BF), (n(E, N, H) * 0.05).to(BF)
    routes = mok.Routes(T, E, K)

    def step():
        sched = routes.build(ids, wts)
        wq, wt = mok.fp8_quantize_weight(w, transposed=True)
        a, at = mok.dispatch_fp8(sched, x, transposed=True)
        y = mok.fp8_grouped_matmul(sched, a, wq)
        out = mok.combine(sched, y)
        dr, dwts = mok.combine_backward(sched, y, dout)
        d, dt = mok.fp8_quantize(dr, transposed=True, sched=sched)
        dx = mok.dispatch_backward(sched, mok.fp8_grouped_matmul(sched, d, wt))
        return out, dwts, dx, mok.fp8_grouped_wgrad(sched, dt, at)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i, kind in enumerate(("few", "spread", "one", "invalid")):
        new_ids, new_w = routing(kind, T, E, K, seed=5 + i)
        ids.copy_(new_ids), wts.copy_(new_w), x.copy_(n(T, H)), dout.copy_(n(T, N)), w.copy_(n(E, N, H) * 0.05)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, step()):
            assert torch.isfinite(a.float()).all() and torch.equal(a, b)
