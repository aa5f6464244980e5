"""Routed rows and 8-bit products at the ends of their ranges, on the GPU vs tests/fp8_ref.py: the most rows, long sums, wide
outputs, one expert (tests/test_gpu_fp8.py and tests/test_gpu_route.py have the tolerances)."""
import pytest
import torch

import fp8_ref as ref
from test_gpu_fp8 import both, codes, near, same, same_scales
from test_gpu_route import EPS, gen, routing

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def test_most_rows(mok):
    """As many rows as a quantisation takes, of the least width; and sums over them."""
    M, K, N = 65535 * 128, 8, 8
    _, n = gen(1)
    x, w = n(M, K).to(BF), codes(N, K, 2, block=True, mok=mok)
    a, at = mok.fp8_quantize(x, transposed=True)
    for rows in (slice(0, 1000), slice(M - 1000, M)):
        q, s = ref.quantize(x[rows], (1, 128))
        same(a.q[rows, :K].contiguous(), q)
        same_scales(a.s[:, rows].T, s)
    assert (a.q[:, K:] == 0).all()
    q, s = ref.quantize(x[-1280:], (128, 1))
    same(at.q[:, -1280:].contiguous(), q.T)
    same_scales(at.s[-10:], s)
    want, mag = both(ref.of(a), ref.of(w))
    near(mok.fp8_linear(x, w), want, mag, 1)
    near(mok.fp8_matmul(a, w, out_dtype=F32), want, mag, 1)
    del want, mag
    full = ref.decode(at.q) * at.s.to(F64).repeat_interleave(128, 0).T
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    near(mok.fp8_matmul(at, at, out_dtype=F32, status=status), *both(full, full), 65535)
    assert int(status) == 0
    with pytest.raises(mok.MokError) as e:
        mok.fp8_linear(torch.zeros((M + 1, K), dtype=BF, device="cuda"), w)
    assert e.value.code == mok.MOK_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,N,K", [(1, 8, 1_000_000), (7, 136, 262_152), (40, 8, 1_000_000), (200, 64, 500_008), (1, 1_000_000, 8), (30, 1_000_000, 136),
                                   (300, 400_000, 8)])
def test_long_sums_and_wide_outputs(mok, M, N, K):
    _, n = gen(M)
    x = n(M, K).to(BF)
    a, _ = mok.fp8_quantize(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for block in (True, False):
        w = codes(N, K, 3, block=block, mok=mok)
        want, mag = both(ref.of(a), ref.of(w))
        near(mok.fp8_matmul(a, w, out_dtype=F32, status=status), want, mag, -(-K // 128))
        if block:
            near(mok.fp8_linear(x, w, status=status), want, mag, -(-K // 128))
    assert int(status) == 0


@pytest.mark.parametrize("T,E,K,H,N", [(1, 1, 1, 8, 8), (3, 1, 1, 136, 264), (47, 1, 1, 264, 136), (48, 1, 1, 264, 136), (500, 1, 1, 520, 72), (5, 2, 2, 8, 16)])
def test_one_expert(mok, T, E, K, H, N):
    ids, w = routing("spread", T, E, K)
    sched = mok.Routes(T, E, K).build(ids, w)
    row, segments, end = ref.layout(ids, E)
    R = sched.c.rpad_max
    _, n = gen(T)
    x, dout, we = n(T, H).to(BF), n(T, N).to(BF), codes(N, H, 1, block=True, batch=E, mok=mok)
    a, at = mok.dispatch_fp8(sched, x, transposed=True)
    y = mok.fp8_grouped_matmul(sched, a, we, out=torch.zeros((R, N), dtype=BF, device="cuda"))
    out, (dr, dw) = mok.combine(sched, y), mok.combine_backward(sched, y, dout)
    d, dt = mok.fp8_quantize(dr, transposed=True, sched=sched)
    grad = mok.fp8_grouped_wgrad(sched, dt, at)
    ax = ref.values(ref.decode(a.q)[:, :H], a.s[:, :a.rows].T, (1, 128))
    axt, adt = (ref.values(ref.decode(m.q)[:, :R], m.s[:, :m.rows].T, (1, 128)) for m in (at, dt))
    for e, (r0, rn) in enumerate(segments):
        if rn:
            near(y[r0:r0 + rn], *both(ax[r0:r0 + rn], ref.of(we, e)), -(-H // 128))
            near(grad[e], *both(adt[:, r0:r0 + rn], axt[:, r0:r0 + rn]), -(-rn // 128))
    want, mag = ref.combine(y, row, w)
    assert ((out.to(F64) - want).abs() <= 2.0**-8 * want.abs() + 2 * K * EPS * mag).all()
    drows, dweights, mag = ref.combine_grads(y, dout, row, w)
    assert ((dr[:end].to(F64) - drows[:end]).abs() <= (2.0**-8 + EPS) * drows[:end].abs()).all()
    assert ((dw.to(F64) - dweights).abs() <= (N + 1) * EPS * mag).all()
    assert mok.mok_read_device_status(sched) == 0
