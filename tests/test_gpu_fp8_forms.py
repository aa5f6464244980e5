"""Routed rows and 8-bit products in the forms that a program calls them: on other streams, behind a slow kernel, from several
threads, at addresses past 32 bits, again and again, and in every tile width (tests/test_gpu_fp8.py has the tolerances)."""
import threading

import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import both, codes, near
from test_gpu_route import gen, routing
from test_gpu_slow_predecessor import hold  # noqa: F401  (a fixture)
from test_streams import owner

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


# wide tiles of the pairs, several rounds of them, more K blocks than a lot of scales; narrow ones; both scalings
@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("M,N,K", [(2600, 2056, 392), (2600, 4104, 5000), (3000, 264, 4360), (300, 5000, 136), (200, 136, 9000)])
def test_widths_rounds_and_long_sums(mok, M, N, K, block):
    a, b = codes(M, K, M + N, mok=mok), codes(N, K, K, block=block, mok=mok)
    want, mag = both(ref.of(a), ref.of(b))
    for dt in (F32, BF):
        got = mok.fp8_matmul(a, b, out_dtype=dt)
        near(got, want, mag, -(-K // 128), dt)
        assert torch.equal(got, mok.fp8_matmul(a, b, out_dtype=dt))


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N,H", [(1000, 1032), (264, 2056), (1024, 512)])
def test_weight_gradients_of_uneven_experts(mok, N, H, dt):
    """Many tiles of a K block or two beside one expert's of sixteen, and of experts without rows: tiles that are taken in turn
    end out of step."""
    T, E, K = 2500, 24, 2
    _, n = gen(N)
    ids = torch.stack([torch.where(torch.arange(T) < 2000, 0, 1 + torch.arange(T) % 9), 10 + torch.arange(T) * 7 % 11], 1)
    ids = ids.to(device="cuda", dtype=torch.int32)
    sched = mok.Routes(T, E, K).build(ids, torch.ones((T, K), device="cuda"))
    _, segments, _ = ref.layout(ids, E)
    assert segments[0][1] == 2000 and segments[-1][1] == 0
    _, at = mok.dispatch_fp8(sched, n(T, H).to(BF), transposed=True, rows=False)
    _, dt_ = mok.fp8_quantize(n(sched.c.rpad_max, N).to(BF), transposed=True, rows=False, sched=sched)
    R = sched.c.rpad_max
    dw = mok.fp8_grouped_wgrad(sched, dt_, at, out_dtype=dt)
    av, xv = (ref.values(ref.decode(m.q)[:, :R], m.s[:, :m.rows].T, (1, 128)) for m in (dt_, at))
    for e, (r0, rn) in enumerate(segments):
        if rn:
            near(dw[e], *both(av[:, r0:r0 + rn], xv[:, r0:r0 + rn]), -(-rn // 128), ("dw", e))
        else:
            assert (dw[e] == 0).all()
    for _ in range(3):
        assert torch.equal(dw, mok.fp8_grouped_wgrad(sched, dt_, at, out_dtype=dt))
    assert mok.mok_read_device_status(sched) == 0


@pytest.mark.parametrize("M", range(1, 18))
def test_few_rows(mok, M):
    """Around the numbers of rows at which a linear takes another way."""
    _, n = gen(M)
    x, w = n(M, 1032).to(BF), codes(264, 1032, 2, block=True, mok=mok)
    a, _ = mok.fp8_quantize(x)
    near(mok.fp8_linear(x, w), *both(ref.of(a), ref.of(w)), 9)


def test_sublayer_shaped_step_on_a_given_stream(mok):
    """Every call on a stream that is not the current one: results as on the current one, allocations owned by that stream."""
    T, E, K, H, N = 150, 5, 2, 264, 392
    ids, wt = routing("spread", T, E, K)
    _, n = gen(3)
    x, w, dy = n(T, H).to(BF), (n(E, N, H) * 0.05).to(BF), n(T, N).to(BF)
    dense = (n(N, H) * 0.05).to(BF)

    def step(s):
        sched = mok.Routes(T, E, K).build(ids, wt, stream=s)
        wq, wqt = mok.fp8_quantize_weight(w, transposed=True, stream=s)
        a, at = mok.dispatch_fp8(sched, x, transposed=True, stream=s)
        y = mok.fp8_grouped_matmul(sched, a, wq, stream=s)
        out = mok.combine(sched, y, stream=s)
        dr, dwt = mok.combine_backward(sched, y, dy, stream=s)
        d, dt = mok.fp8_quantize(dr, transposed=True, sched=sched, stream=s)
        dx = mok.dispatch_backward(sched, mok.fp8_grouped_matmul(sched, d, wqt, stream=s), stream=s)
        dw = mok.fp8_grouped_wgrad(sched, dt, at, stream=s)
        rows = mok.dispatch(sched, x, stream=s)
        lw, _ = mok.fp8_quantize_weight(dense, stream=s)
        lin, few = mok.fp8_linear(x, lw, stream=s), mok.fp8_linear(x[:3], lw, stream=s)
        q, qt = mok.fp8_quantize(x, transposed=True, stream=s)
        mm = mok.fp8_matmul(q, lw, stream=s)
        end = int(sched.tables()["poff"][E]) if s is None else None
        return sched, end, [out, dwt, dx, dw, lin, few, mm, y, dr, rows, wq.q, wq.s, a.q, at.s, q.q, qt.q, qt.s]
    sched, end, want = step(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    sched2, _, got = step(side)
    assert torch.cuda.current_stream() != side
    for t in got:
        assert owner(t) == side.cuda_stream
    torch.cuda.synchronize()
    assert mok.mok_read_device_status(sched2) == 0
    for a, b in zip(got[:7], want[:7]):
        assert torch.equal(a, b)
    for a, b in zip(got[8:10], want[8:10]):
        assert torch.equal(a[:end], b[:end])


def test_no_wait_counts_while_the_kernel_in_front_runs(mok, hold):  # noqa: F811
    """Behind a kernel that lets its successor start and then runs for longer than any wait inside a kernel may."""
    stream = torch.cuda.current_stream().cuda_stream
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for M, N, K in ((3, 264, 1032), (40, 264, 1032), (1500, 1032, 520)):
        _, n = gen(M)
        x, w = n(M, K).to(BF), codes(N, K, 1, block=True, mok=mok)
        a, at = mok.fp8_quantize(x, transposed=True)
        run = [lambda: mok.fp8_linear(x, w, status=status), lambda: mok.fp8_matmul(a, w, status=status),  # noqa: B023
               lambda: mok.fp8_matmul(at, at, status=status)]  # noqa: B023
        want = [f() for f in run]
        for f, y in zip(run, want):
            torch.cuda.synchronize()
            assert hold(stream) == 0
            assert torch.equal(f(), y)
    ids, wt = routing("spread", 600, 4, 2)
    sched = mok.Routes(600, 4, 2).build(ids, wt)
    _, n = gen(1)
    x, w = n(600, 264).to(BF), codes(136, 264, 2, block=True, batch=4, mok=mok)
    a, at = mok.dispatch_fp8(sched, x, transposed=True)
    run = [lambda: mok.fp8_grouped_matmul(sched, a, w, out=torch.zeros((sched.c.rpad_max, 136), dtype=BF, device="cuda")),
           lambda: mok.fp8_grouped_wgrad(sched, at, at)]
    want = [f() for f in run]
    for f, y in zip(run, want):
        torch.cuda.synchronize()
        assert hold(stream) == 0
        assert torch.equal(f(), y)
    assert int(status) == 0 and mok.mok_read_device_status(sched) == 0


def test_weights_quantised_right_before(mok):
    """A product behind the kernel that writes its weights: it does not read them early."""
    for M in (2, 40, 700):
        _, n = gen(M)
        x, w = n(M, 2056).to(BF), n(1032, 2056).to(BF)
        want = mok.fp8_linear(x, mok.fp8_quantize_weight(w)[0])
        buf = mok.fp8_quantize_weight(torch.zeros_like(w))[0]
        L, stream = mok._lib, torch.cuda.current_stream().cuda_stream
        out = torch.empty_like(want)
        for _ in range(20):
            buf.q.zero_(), buf.s.zero_()
            assert L.mok_fp8_quantize_blocks(w.data_ptr(), 1, 1032, 2056, buf.q.data_ptr(), buf.s.data_ptr(), None, None, stream) == 0
            assert torch.equal(mok.fp8_linear(x, buf, out=out), want)


def test_from_several_threads(mok):
    """Calls of several threads at once, each on a stream of its own."""
    T, E, K, H, N = 200, 6, 2, 264, 136
    _, n = gen(4)
    x, w = n(T, H).to(BF), codes(N, H, 1, block=True, batch=E, mok=mok)
    lw = codes(N, H, 2, block=True, mok=mok)
    routings = [routing("spread", T, E, K, seed=i) for i in range(4)]

    def step(i, s):
        sched = mok.Routes(T, E, K).build(*routings[i], stream=s)
        a, _ = mok.dispatch_fp8(sched, x, stream=s)
        return mok.combine(sched, mok.fp8_grouped_matmul(sched, a, w, stream=s), stream=s), mok.fp8_linear(x, lw, stream=s)
    want = [step(i, None) for i in range(4)]
    torch.cuda.synchronize()
    bad = []

    def worker(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got = step(i, s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)
    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_other_threads_run_while_a_launch_waits(mok):
    """3000 calls behind about a second of GPU work: more launches than the queue holds, so that some wait."""
    import time
    x, w = torch.ones((1, 64), dtype=BF, device="cuda"), codes(16, 64, 1, block=True, mok=mok)
    mok.fp8_linear(x, w)
    torch.cuda.synchronize()
    stop, ticks = threading.Event(), []

    def tick():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.monotonic()
            ticks.append(now - last)
            last = now
    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(2_000_000_000)
        longest = 0.0
        for _ in range(3000):
            t0 = time.monotonic()
            mok.fp8_linear(x, w)
            longest = max(longest, time.monotonic() - t0)
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    assert longest < 0.05 or max(ticks) < longest / 2, (longest, max(ticks))


def test_addresses_past_32_bits(mok):
    """600,000 rows of 4096: codes, routed rows and outputs of more than 2^31 values; their last rows are right."""
    T, K, W = 75_000, 8, 4096
    g, n = gen(5)
    x = n(T, W).to(BF)
    ids, wt = torch.zeros((T, K), dtype=torch.int32, device="cuda"), torch.rand((T, K), generator=g, device="cuda")
    sched = mok.Routes(T, 8, K).build(ids, wt)
    rows = mok.dispatch(sched, x)
    tail = slice(T * K - 400, T * K)
    token = torch.arange(T * K, device="cuda")[tail] // K
    assert torch.equal(rows[tail], x[token]) and torch.equal(rows[:400], x[torch.arange(400, device="cuda") // K])
    w = codes(W, W, 6, block=True, batch=8, mok=mok)
    a, at = mok.dispatch_fp8(sched, x, transposed=True)
    small, _ = mok.fp8_quantize(x[token])
    assert torch.equal(a.q[tail], small.q) and torch.equal(a.s[:, tail], small.s)
    y = mok.fp8_grouped_matmul(sched, a, w, out=rows)
    near(y[tail], *both(ref.of(small), ref.of(w, 0)), W // 128)
    only, _ = mok.dispatch_fp8(sched, x)
    assert torch.equal(only.q[tail], small.q)
    del only
    assert torch.equal(at.q[:, T * K - 400:T * K][:64], mok.fp8_quantize(x[(torch.arange(T * K, device="cuda")[T * K // 128 * 128 - 512:]) // K],
                                                                        rows=False, transposed=True)[1].q[:64, 512 - 400 + T * K % 128:512 + T * K % 128])
    out = mok.combine(sched, y)
    want = (y[tail].view(-1, K, W).to(F64) * wt[token[0]:, :, None].to(F64)).sum(1)
    mag = (y[tail].view(-1, K, W).to(F64) * wt[token[0]:, :, None].to(F64)).abs().sum(1)
    assert ((out[token[0]:].to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * 2.0**-24 * mag).all()
    yc = y[tail].clone()
    dr, dw = mok.combine_backward(sched, y, x, drows=y)
    want = x[token].to(F64) * wt.flatten()[tail, None].to(F64)
    assert ((dr[tail].to(F64) - want).abs() <= (2.0**-8 + 2.0**-24) * want.abs()).all()
    p = yc.to(F64) * x[token].to(F64)
    assert ((dw.flatten()[tail].to(F64) - p.sum(1)).abs() <= (W + 1) * 2.0**-24 * p.abs().sum(1)).all()
    dense = mok.Fp8(a.q[:T * K], a.s[:, :T * K].contiguous(), W)
    w0 = mok.Fp8(w.q[0], w.s[0], W, True)
    near(mok.fp8_matmul(dense, w0, out=rows[:T * K])[tail], *both(ref.of(small), ref.of(w0)), W // 128)


@pytest.mark.parametrize("kind", ["one", "few", "spread", "invalid"])
def test_again_and_again(mok, kind):
    """Bits do not change from run to run, whatever ran before; two schedules on workspaces of their own do not meet."""
    T, E, K, H, N = 700, 9, 3, 520, 392
    _, n = gen(7)
    x, w = n(T, H).to(BF), codes(N, H, 1, block=True, batch=E, mok=mok)
    r = [mok.Routes(T, E, K) for _ in range(2)]
    s = [r[i].build(*routing(kind, T, E, K, seed=i)) for i in range(2)]

    def step(s):
        a, at = mok.dispatch_fp8(s, x, transposed=True)
        y = mok.fp8_grouped_matmul(s, a, w, out=torch.zeros((s.c.rpad_max, N), dtype=BF, device="cuda"))
        return y, mok.combine(s, y), mok.fp8_grouped_wgrad(s, at, at)
    want = [step(v) for v in s]
    for _ in range(5):
        for v, y in zip(s, want):
            assert all(torch.equal(p, q) for p, q in zip(step(v), y))
