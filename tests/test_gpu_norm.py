"""Norm of the residual stream and dropout on the GPU vs the 64-bit formulas (tests/dense_ref.py).

Tolerances, from the arithmetic: a bf16 output is rounded once, 2^-8 of its value at most (half of a
2^-7 step), an fp32 output carries a few fp32 roundings; sums of n fp32 terms in chains and trees of at
most 64 stay within 2^-24 * 64 of the sum of their magnitudes, taken here as REL = 1e-5.  The norm is
checked from the stream h the kernel stored, the backward from the rstd the forward stored.
"""
import numpy as np
import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
REL = 1e-5
SEED, OFFSET = -0x123456789ABCDEF, 0x1_0000_0007  # the state's words are bit patterns


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def rng_state(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def near(got, want, scale=None, name=""):
    """got (bf16 or fp32) within one rounding plus REL of `scale` (defaults to |want|)."""
    got, want = got.detach().cpu(), want
    mag = want.abs() if scale is None else scale
    tol = (2.0**-8 if got.dtype == BF else 0.0) * want.abs() + REL * mag + 1e-30
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), name
    assert (err <= tol).all(), (name, float((err / tol).max()))


def draw(T, H, stream, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(x=n(T, H).to(BF), res=(2 * n(T, H)).to(stream), w=(1 + 0.1 * n(H)).to(BF), dy=n(T, H).to(BF),
                dres=n(T, H).to(stream))


def check_mx(q, s, y):
    """Codes and scales against the unrounded rows: the scale is floor(log2 max) - 8 of the block (either
    neighbour when the maximum is within REL of a power of two) and every code the nearest E4M3 value."""
    T, H = y.shape
    v = y.view(T, H // 32, 32)
    top = v.abs().amax(2)
    e = s.cpu().int() - 127
    lo, hi = torch.floor(torch.log2(top * (1 - REL))) - 8, torch.floor(torch.log2(top * (1 + REL))) - 8
    zero = top == 0
    assert ((e == lo) | (e == hi) | (zero & (e == -127))).all()
    scaled = (v * torch.exp2(-e.double())[:, :, None]).clamp(-448, 448)
    code = q.cpu().view(torch.float8_e4m3fn).double().view(v.shape)
    step = torch.exp2(torch.floor(torch.log2(scaled.abs().clamp(min=2.0**-6))) - 3)
    assert ((code - scaled).abs() <= 0.5 * step + REL * scaled.abs() + 1e-30).all()


CASES = [(1, 8, BF, 0.0), (1, 4096, BF, 0.1), (3, 64, F32, 0.0), (17, 96, BF, 0.5), (5, 264, F32, 0.1), (33, 2048, BF, 0.0),
         (40, 2056, F32, 0.3), (700, 1024, BF, 0.1), (31, 7168, BF, 0.2), (9, 8200, F32, 0.1), (7, 16384, BF, 0.1),
         (6, 16384, F32, 0.0), (2500, 128, BF, 0.1)]


@pytest.mark.parametrize("T,H,stream,p", CASES)
def test_norm_forward_and_backward(mok, T, H, stream, p):
    d = draw(T, H, stream, T + H)
    c = {k: v.cuda() for k, v in d.items()}
    state = rng_state()
    drop = mok.Dropout(p, state) if p else None
    mx = H % 32 == 0
    o = mok.rmsnorm_forward(c["x"], c["w"], 1e-5, residual=c["res"], dropout=drop, mx=mx)
    f = lambda v: ref.dropped(v, p, SEED, OFFSET) if p else v  # noqa: E731
    xd = f(d["x"].double())
    near(o.h, d["res"].double() + xd, d["res"].double().abs() + xd.abs(), "h")
    assert o.h.dtype == stream
    h = o.h.cpu().double()
    y, rstd = ref.rmsnorm(h, d["w"].double(), 1e-5)
    near(o.rstd, rstd, name="rstd")
    near(o.y, y, name="y")
    if mx:
        check_mx(o.q, o.s, y)
        only = mok.rmsnorm_forward(c["x"], c["w"], 1e-5, residual=c["res"], dropout=drop, bf16=False, mx=True)
        assert only.y is None and torch.equal(only.q, o.q) and torch.equal(only.s, o.s) and torch.equal(only.h, o.h)
    for dres in (c["dres"], None):
        g = mok.rmsnorm_backward(o.h, o.rstd, c["w"], c["dy"], dres=dres, dropout=drop)
        dr = None if dres is None else d["dres"].double()
        dy, w, rs = d["dy"].double(), d["w"].double(), o.rstd.cpu().double()
        dh, dw = ref.rmsnorm_grads(h, rs, w, dy, dr)
        xh = (h * rs[:, None]).abs()
        mag = rs[:, None] * ((dy * w).abs() + xh * ((dy * w).abs() * xh).mean(1, keepdim=True))
        mag = mag if dr is None else mag + dr.abs()
        near(g.dh, dh, mag, "dh")
        near(g.dx, f(dh), f(mag) if p else mag, "dx")
        near(g.dweight, dw, (dy.abs() * xh).sum(0), "dweight")


def test_norm_without_residual_or_dropout_keeps_x(mok):
    d = draw(19, 512, BF, 3)
    x, w = d["x"].cuda(), d["w"].cuda()
    o = mok.rmsnorm_forward(x, w, 1e-6)
    assert o.h is x
    near(o.y, ref.rmsnorm(d["x"].double(), d["w"].double(), 1e-6)[0], name="y")
    state = rng_state()
    o = mok.rmsnorm_forward(x, w, 1e-6, dropout=mok.Dropout(0.25, state))  # h = dropout(x)
    near(o.h, ref.dropped(d["x"].double(), 0.25, SEED, OFFSET), name="h")


@pytest.mark.parametrize("stream", [BF, F32])
def test_in_place_stream_and_gradient(mok, stream):
    d = draw(50, 1032, stream, 4)
    c = {k: v.cuda() for k, v in d.items()}
    state = rng_state()
    drop = mok.Dropout(0.1, state)
    want = mok.rmsnorm_forward(c["x"], c["w"], 1e-6, residual=c["res"], dropout=drop)
    wg = mok.rmsnorm_backward(want.h, want.rstd, c["w"], c["dy"], dres=c["dres"], dropout=drop)
    import ctypes
    shape = mok.mok_norm_shape(50, 1032, 0 if stream == BF else 1, 1e-6)
    h, y, rstd = c["res"].clone(), torch.empty_like(c["x"]), torch.empty(50, device="cuda")
    rc = mok._lib.mok_rmsnorm_forward(ctypes.byref(shape), c["x"].data_ptr(), h.data_ptr(), drop.ref, c["w"].data_ptr(),
                                      h.data_ptr(), y.data_ptr(), None, None, rstd.data_ptr(), mok._stream(None))
    assert rc == 0 and torch.equal(h, want.h) and torch.equal(y, want.y)
    dh, dx, dw = c["dres"].clone(), c["dy"].clone(), torch.empty(1032, device="cuda")
    ws = torch.empty(mok.mok_rmsnorm_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    rc = mok._lib.mok_rmsnorm_backward(ctypes.byref(shape), h.data_ptr(), rstd.data_ptr(), c["w"].data_ptr(), dx.data_ptr(),
                                       dh.data_ptr(), drop.ref, dh.data_ptr(), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                                       ws.numel(), mok._stream(None))
    assert rc == 0 and torch.equal(dh, wg.dh) and torch.equal(dx, wg.dx) and torch.equal(dw, wg.dweight)


def test_rows_of_zeros_infinities_and_nan_stay_their_own(mok):
    d = draw(8, 256, F32, 5)
    x, res = torch.zeros_like(d["x"]), d["res"].clone()
    res[1] = 0.0                         # rstd = eps^-1/2, y = 0
    res[3, 17] = float("nan")
    res[5, 40] = float("inf")
    o = mok.rmsnorm_forward(x.cuda(), d["w"].cuda(), 1e-6, residual=res.cuda(), mx=True)
    y = o.y.cpu().float()
    assert (y[1] == 0).all() and abs(o.rstd[1].item() - 1e3) < 1e-2 and (o.q[1] == 0).all() and (o.s[1] == 0).all()
    assert torch.isnan(y[3]).all() and (o.s[3] == 255).all() and (o.q[3] == 0x7F).all()
    assert torch.isnan(y[5, 40]) and (y[5, :32] == 0).all() and o.s[5, 1] == 255 and (o.q[5, 32:64] == 0x7F).all()
    ok = [0, 2, 4, 6, 7]
    near(o.y[ok], ref.rmsnorm(res[ok].double(), d["w"].double(), 1e-6)[0], name="y")


def test_no_rows(mok):
    e = torch.empty((0, 64), dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    o = mok.rmsnorm_forward(e, w, 1e-6, residual=e, mx=True)
    assert o.y.shape == (0, 64)
    g = mok.rmsnorm_backward(e, o.rstd, w, e)
    assert (g.dweight == 0).all()
    state = rng_state()
    assert mok.dropout_forward(e, mok.Dropout(0.5, state)).numel() == 0


@pytest.mark.parametrize("T,H,stream,p", [(32, 128, BF, 0.1), (64, 512, F32, 0.0), (6, 1024, BF, 0.1), (34, 2048, BF, 0.1),
                                          (5, 4096, BF, 0.1), (4, 2048, F32, 0.1), (3, 7168, BF, 0.0), (3, 8192, F32, 0.1)])
def test_rows_do_not_depend_on_how_many_there_are(mok, T, H, stream, p):
    """T rows that fill every block and T + 1 that do not give the first T the same bits; in place as well."""
    d = draw(T + 1, H, stream, 3 * T + H)
    c = {k: v.cuda() for k, v in d.items()}
    state = rng_state()
    drop = mok.Dropout(p, state) if p else None
    o = mok.rmsnorm_forward(c["x"], c["w"], 1e-5, residual=c["res"], dropout=drop, mx=True)
    g = mok.rmsnorm_backward(o.h, o.rstd, c["w"], c["dy"], dres=c["dres"], dropout=drop)
    cut = {k: v[:T].clone() if v.dim() == 2 else v for k, v in c.items()}
    a = mok.rmsnorm_forward(cut["x"], cut["w"], 1e-5, residual=cut["res"], dropout=drop, mx=True)
    b = mok.rmsnorm_backward(a.h, a.rstd, cut["w"], cut["dy"], dres=cut["dres"], dropout=drop)
    for k in "h", "rstd", "y", "q", "s":
        assert torch.equal(getattr(a, k), getattr(o, k)[:T]), k
    assert torch.equal(b.dh, g.dh[:T]) and torch.equal(b.dx, g.dx[:T])
    h = a.h.cpu().double()
    _, dw = ref.rmsnorm_grads(h, a.rstd.cpu().double(), d["w"].double(), d["dy"][:T].double(), None)
    near(b.dweight, dw, (d["dy"][:T].double().abs() * (h * a.rstd.cpu().double()[:, None]).abs()).sum(0), "dweight")
    import ctypes
    shape = mok.mok_norm_shape(T, H, 0 if stream == BF else 1, 1e-5)
    dh, dx, dweight = cut["dres"].clone(), cut["dy"].clone(), torch.empty(H, device="cuda")
    ws = torch.empty(mok.mok_rmsnorm_workspace_bytes(shape), dtype=torch.uint8, device="cuda")
    rc = mok._lib.mok_rmsnorm_backward(ctypes.byref(shape), a.h.data_ptr(), a.rstd.data_ptr(), c["w"].data_ptr(),
                                       dx.data_ptr(), dh.data_ptr(), drop.ref if drop else None, dh.data_ptr(),
                                       dx.data_ptr(), dweight.data_ptr(), ws.data_ptr(), ws.numel(), mok._stream(None))
    assert rc == 0 and torch.equal(dh, b.dh) and torch.equal(dx, b.dx) and torch.equal(dweight, b.dweight)


@pytest.mark.parametrize("n,stream,p", [(8, BF, 0.5), (8 * 511, F32, 0.1), (8 * 513, BF, 0.1), (8 * 40001, BF, 0.02),
                                        (8 * 1000, F32, 0.0), (8 * 1000, BF, 1.0)])
def test_dropout(mok, n, stream, p):
    g = torch.Generator().manual_seed(n)
    x, res = torch.randn(n, generator=g).to(BF), torch.randn(n, generator=g).to(stream)
    x[3] = float("inf")  # a dropped value contributes 0 whatever it holds
    x[5] = float("nan")
    state = rng_state()
    drop = mok.Dropout(p, state)
    clean = torch.nan_to_num(x.float(), nan=1.0, posinf=1.0).double()
    bad = ref.dropped((~torch.isfinite(x.float())).double(), p, SEED, OFFSET) != 0
    for r in (res, None):
        out = mok.dropout_forward(x.cuda(), drop, residual=None if r is None else r.cuda())
        assert out.dtype == (BF if r is None else stream)
        want = ref.dropped(clean, p, SEED, OFFSET) + (0 if r is None else r.double())
        got = out.cpu()
        assert not torch.isfinite(got[bad].float()).any()
        near(torch.where(bad, want.to(got.dtype), got), want, want.abs() + clean.abs() * 2, "out")
    dout = torch.randn(n, generator=g).to(stream)
    near(mok.dropout_backward(dout.cuda(), drop), ref.dropped(dout.double(), p, SEED, OFFSET), name="dx")
    inplace = x.cuda()
    assert torch.equal(mok.dropout_forward(inplace, drop, out=inplace).nan_to_num(),
                       mok.dropout_forward(x.cuda(), drop).nan_to_num())


def test_state_is_read_when_the_kernel_runs(mok):
    x = torch.ones((64, 512), dtype=BF, device="cuda")
    state = rng_state(5, 0)
    drop = mok.Dropout(0.5, state)
    a = mok.dropout_forward(x, drop)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(x)
    with torch.cuda.graph(g):
        mok.dropout_forward(x, drop, out=out)
        state[1] += 1
    masks = []
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        masks.append(out.clone())
        assert torch.equal(out.cpu() != 0, ref.keep((64, 512), 0.5, 5, i))
    assert torch.equal(masks[0], a) and not torch.equal(masks[1], masks[0])


def test_side_stream_repeats_and_offsets_past_32_bits(mok):
    H, T = 8192, 300_000  # 2.46 G values
    x = torch.empty((T, H), dtype=BF, device="cuda").normal_()
    w = torch.ones(H, dtype=BF, device="cuda")
    state = rng_state()
    drop = mok.Dropout(0.1, state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = mok.rmsnorm_forward(x, w, 1e-6, dropout=drop)
        g = mok.rmsnorm_backward(o.h, o.rstd, w, x, dropout=drop)
        d = mok.dropout_forward(x.view(-1), drop)
    side.synchronize()
    rows = slice(T - 3, T)
    n = 3 * H
    kept = torch.from_numpy(ref.draws16(n, SEED, OFFSET, (T - 3) * H // 8) >= ref.threshold(0.1)).view(3, H)
    xt = x[rows].cpu().double()
    want = torch.where(kept, xt * (65536 / (65536 - ref.threshold(0.1))), torch.zeros_like(xt))
    near(o.h[rows], want, name="h")
    near(d.view(T, H)[rows], want, name="dropout")
    h = o.h[rows].cpu().double()
    near(o.y[rows], ref.rmsnorm(h, w.cpu().double(), 1e-6)[0], name="y")
    again = mok.rmsnorm_backward(o.h, o.rstd, w, x, dropout=drop)
    assert torch.equal(again.dweight, g.dweight) and torch.equal(again.dx, g.dx) and torch.equal(again.dh, g.dh)
    assert np.isfinite(g.dweight.double().sum().item())


@pytest.mark.parametrize("handle", [False, True])
def test_a_given_stream_owns_what_the_call_allocates(mok, handle):
    d = draw(300, 1032, BF, 9)
    c = {k: v.cuda() for k, v in d.items()}
    drop = mok.Dropout(0.1, rng_state())
    want = mok.rmsnorm_forward(c["x"], c["w"], 1e-6, residual=c["res"], dropout=drop)
    wg = mok.rmsnorm_backward(want.h, want.rstd, c["w"], c["dy"], dres=c["dres"], dropout=drop)
    wd, wb = mok.dropout_forward(c["x"], drop, residual=c["res"]), mok.dropout_backward(c["dres"], drop)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    o = mok.rmsnorm_forward(c["x"], c["w"], 1e-6, residual=c["res"], dropout=drop, stream=s)
    g = mok.rmsnorm_backward(want.h, want.rstd, c["w"], c["dy"], dres=c["dres"], dropout=drop, stream=s)
    f, b = mok.dropout_forward(c["x"], drop, residual=c["res"], stream=s), mok.dropout_backward(c["dres"], drop, stream=s)
    assert torch.cuda.current_stream() != side
    pools = torch.cuda.memory_snapshot()  # each segment with the stream that owns it
    for t in (o.h, o.y, o.rstd, g.dh, g.dx, g.dweight, f, b):
        owner = [p["stream"] for p in pools if p["address"] <= t.data_ptr() < p["address"] + p["total_size"]]
        assert owner == [side.cuda_stream]
    torch.cuda.synchronize()
    assert torch.equal(o.h, want.h) and torch.equal(o.y, want.y) and torch.equal(o.rstd, want.rstd)
    assert torch.equal(g.dh, wg.dh) and torch.equal(g.dx, wg.dx) and torch.equal(g.dweight, wg.dweight)
    assert torch.equal(f, wd) and torch.equal(b, wb)


def test_wrong_tensors_are_named(mok):
    d = draw(16, 64, BF, 2)
    c = {k: v.cuda() for k, v in d.items()}
    x, res, w, dy = c["x"], c["res"], c["w"], c["dy"]
    drop = mok.Dropout(0.1, rng_state())
    rstd = torch.ones(16, device="cuda")
    turned = x.t().contiguous().t()
    for bad, name in ((dict(x=turned), "x"), (dict(x=x.float()), "x"), (dict(x=x.cpu()), "x"), (dict(weight=w[:32]), "weight"),
                      (dict(weight=w.float()), "weight"), (dict(residual=res[:8]), "residual"),
                      (dict(residual=res.half()), "residual"), (dict(residual=turned), "residual"), (dict(weight=None), "weight")):
        with pytest.raises(ValueError, match=name):
            mok.rmsnorm_forward(**{**dict(x=x, weight=w, eps=1e-6, residual=res), **bad})
    for bad, name in ((dict(h=x.half()), "h"), (dict(rstd=rstd[:8]), "rstd"), (dict(rstd=rstd.double()), "rstd"),
                      (dict(weight=w.float()), "weight"), (dict(dy=turned), "dy"), (dict(dy=dy.float()), "dy"),
                      (dict(dres=dy.float()), "dres"), (dict(h=turned), "h")):
        with pytest.raises(ValueError, match=name):
            mok.rmsnorm_backward(**{**dict(h=x, rstd=rstd, weight=w, dy=dy, dres=res), **bad})
    for call in (lambda: mok.dropout_forward(x.float(), drop), lambda: mok.dropout_forward(x, drop, residual=res[:8]),
                 lambda: mok.dropout_forward(x, drop, out=torch.empty_like(x, dtype=F32)),
                 lambda: mok.dropout_backward(x.half(), drop), lambda: mok.dropout_backward(x, drop, dx=res.float()),
                 lambda: mok.rmsnorm_forward(x.view(-1), w, 1e-6)):
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros((4, 68), dtype=BF, device="cuda")
    for call in (lambda: mok.rmsnorm_forward(odd, odd[0].clone(), 1e-6), lambda: mok.rmsnorm_forward(x, w, float("nan")),
                 lambda: mok.rmsnorm_forward(c["x"][:, :40].contiguous(), w[:40].clone(), 1e-6, mx=True),
                 lambda: mok.rmsnorm_backward(odd, rstd[:4].clone(), odd[0].clone(), odd),
                 lambda: mok.dropout_forward(torch.zeros(12, dtype=BF, device="cuda"), drop)):
        with pytest.raises(mok.MokError):
            call()
    with pytest.raises(TypeError):
        mok.rmsnorm_forward(x, w, "eps")
