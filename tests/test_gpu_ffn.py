"""The dense gated feed-forward block on the GPU vs the 64-bit formulas (tests/dense_ref.py).

Tolerances, element by element, from the roundings the block makes: the inner operand of each second
product (a forward; dg, du backward) is rounded to bf16, 2^-8 of its value at most, so an output moves by
at most 2^-8 of the product of the magnitudes; the output is rounded once more (2^-8 of it, bf16).  fp32
accumulation and the fast exponential and division add a few fp32 ulp of every product's magnitudes
and of g, u: SLACK = 1e-4 of the product of the magnitudes covers K up to 10^4 with |g| <= 20.
"""
import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SLACK = 1e-4


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def draw(T, H, I, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    sc = 1.5 / H**0.5
    d = dict(x=n(T, H), wg=n(I, H) * sc, wu=n(I, H) * sc, wd=n(H, I) * sc, dy=n(T, H))
    d = {k: v.to(BF) for k, v in d.items()}
    d["res"] = n(T, H).to(BF) if residual else None
    return d


def near(got, want, mag, name):
    """mag: product of the magnitudes behind `want` (with the rounded operand)."""
    tol = (2.0**-8 + SLACK) * mag + (2.0**-8 if got.dtype == BF else 0.0) * want.abs() + 1e-30
    err = (got.double() - want).abs()
    assert torch.isfinite(got.float()).all(), name
    assert (err <= tol).all(), (name, float((err / tol).max()))


def check(mok, T, H, I, act, residual=True, train=True, dw_dtype=BF, seed=0, plan=None):
    d = draw(T, H, I, seed + T + H + I, residual)
    plan = plan or mok.FFN(T, H, I, act=act, train=train, dw_dtype=dw_dtype)
    w = (d["wg"], d["wu"], d["wd"])
    out = plan.forward(d["x"], *w, residual=d["res"])
    t = [v.double() for v in (d["x"], *w)]
    want, saved = ref.ffn(*t, act, None if d["res"] is None else d["res"].double())
    a = saved[4]
    near(out, want, a.abs() @ t[3].T.abs() + (0 if d["res"] is None else d["res"].double().abs()), "out")
    if train:
        g = plan.backward(d["x"], *w, d["dy"])
        dy = d["dy"].double()
        r, (dg, du) = ref.ffn_grads(*t, dy, saved)
        # da's own fp32 error scales with the magnitudes of its products, not with da
        da_mag = dy.abs() @ t[3].abs()
        dgm = dg.abs() + 1e-2 * da_mag * saved[1].abs()
        dum = du.abs() + 1e-2 * da_mag * saved[0].abs()
        near(g.dx, r["dx"], dgm @ t[1].abs() + dum @ t[2].abs(), "dx")
        near(g.dw_gate, r["dw_gate"], dgm.T @ t[0].abs(), "dw_gate")
        near(g.dw_up, r["dw_up"], dum.T @ t[0].abs(), "dw_up")
        near(g.dw_down, r["dw_down"], dy.abs().T @ a.abs(), "dw_down")
        assert g.dw_gate.dtype == dw_dtype
    assert plan.device_status() == 0
    return plan, d


@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (1, 256, 128), (1, 4096, 1536), (2, 72, 200), (7, 64, 1000), (8, 2048, 1024),
                                   (61, 520, 264), (64, 1024, 512), (127, 128, 136), (128, 256, 384), (129, 136, 128),
                                   (200, 2056, 72), (255, 512, 2048), (256, 256, 256), (257, 1032, 520),
                                   (513, 768, 640), (1003, 2056, 1000), (2048, 512, 768), (3001, 264, 136)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward_and_gradients(mok, T, H, I, act):
    check(mok, T, H, I, act, residual=act == "silu")


@pytest.mark.parametrize("T", [1, 16, 61, 130, 700])
def test_inference_plan(mok, T):
    check(mok, T, 1024, 768, "silu", train=False)


def test_fp32_weight_gradients(mok):
    check(mok, 300, 264, 200, "silu", dw_dtype=F32)
    check(mok, 2000, 512, 640, "gelu", dw_dtype=F32)


def test_large_tiles(mok):
    check(mok, 8192, 1024, 1536, "silu")
    check(mok, 4100, 2048, 1024, "gelu")


def test_no_tokens(mok):
    d = draw(0, 64, 32, 1)
    plan = mok.FFN(0, 64, 32, dw_dtype=F32)
    assert plan.forward(d["x"], d["wg"], d["wu"], d["wd"], residual=d["res"]).shape == (0, 64)
    g = plan.backward(d["x"], d["wg"], d["wu"], d["wd"], d["dy"])
    assert all((t == 0).all() for t in (g.dw_gate, g.dw_up, g.dw_down))


@pytest.mark.parametrize("T", [1, 5, 130, 600])
def test_bad_tokens_stay_their_own(mok, T):
    """A NaN or an infinity in one token's row reaches that row's output alone, whatever the tile's other
    rows and the shared memory of earlier kernels hold."""
    H, I = 264, 136
    poison = draw(256, H, I, 9)
    poison["x"][:] = float("nan")
    p = mok.FFN(256, H, I)
    p.forward(poison["x"], poison["wg"], poison["wu"], poison["wd"])
    plan, d = check(mok, T, H, I, "silu")
    clean = plan.out.clone()
    if T > 1:
        x = d["x"].clone()
        x[T // 2, 3] = float("nan")
        x[0, 5] = float("inf")
        out = plan.forward(x, d["wg"], d["wu"], d["wd"], residual=d["res"])
        keep = [t for t in range(T) if t not in (0, T // 2)]
        assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[T // 2].float()).any()


def test_repeats_side_stream_graph_and_in_place(mok):
    T, H, I = 300, 520, 264
    plan, d = check(mok, T, H, I, "silu")
    w = (d["wg"], d["wu"], d["wd"])
    first = [plan.out.clone()] + [getattr(plan.grads, k).clone() for k in ("dx", "dw_gate", "dw_up", "dw_down")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            plan.forward(d["x"], *w, residual=d["res"])
            plan.backward(d["x"], *w, d["dy"])
    side.synchronize()
    again = [plan.out] + [getattr(plan.grads, k) for k in ("dx", "dw_gate", "dw_up", "dw_down")]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.forward(d["x"], *w, residual=d["res"])
        plan.backward(d["x"], *w, d["dy"])
    for t in again:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    plan.out.copy_(d["res"])  # the residual's buffer as the output
    assert torch.equal(plan.forward(d["x"], *w, residual=plan.out), first[0])


def test_gradients_left_out(mok):
    import ctypes
    T, H, I = 200, 136, 72
    plan, d = check(mok, T, H, I, "gelu", residual=False)
    want = {k: getattr(plan.grads, k).clone() for k in ("dx", "dw_gate", "dw_up", "dw_down")}
    for keep in (("dx",), ("dw_gate", "dw_up"), ("dw_down",), ()):
        got = {k: torch.zeros_like(v) for k, v in want.items()}
        gr = mok.mok_ffn_grads(*[got[k].data_ptr() if k in keep else None for k in want], 0)
        rc = mok._lib.mok_ffn_backward(ctypes.byref(plan.shape), d["x"].data_ptr(), d["wg"].data_ptr(), d["wu"].data_ptr(),
                                       d["wd"].data_ptr(), plan.ctx.data_ptr(), plan.ctx.numel(), d["dy"].data_ptr(),
                                       ctypes.byref(gr), plan.ws.data_ptr(), plan.ws.numel(), None, mok._stream(None))
        assert rc == 0
        for k in want:
            assert torch.equal(got[k], want[k]) if k in keep else (got[k] == 0).all()


# Sizes by the tile widths of the pair kernel: GATEUP, DOWN, the backward's two launches (- : on the tile kernel).
@pytest.mark.parametrize("T,H,I,widths", [
    (512, 5000, 2600, "192 192 192 256"), (1100, 2048, 1024, "192 192 128 256"), (2048, 4096, 1536, "192 224 224 224"),
    (700, 3400, 3400, "192 192 192 224"), (5120, 1792, 896, "256 256 128 224"), (396, 160, 1584, "128 - 128 128"),
    (580, 1720, 128, "- 128 - 128"), (1662, 192, 2288, "256 - 256 128"), (372, 2792, 136, "- 128 - 192")])
def test_every_tile_width(mok, T, H, I, widths):
    check(mok, T, H, I, "silu" if T % 3 else "gelu")


# Sizes whose GATEUP or DOWN takes two tile widths: the first M tiles in one, the last in the other.
@pytest.mark.parametrize("T,H,I,widths", [
    (1370, 80, 1768, "gate/up 192 128"), (2759, 104, 1272, "gate/up 256 128"), (2078, 88, 1624, "gate/up 256 192"),
    (1300, 3344, 80, "down 192 128"), (3224, 3272, 80, "down 224 128"), (2349, 2968, 80, "down 224 192"),
    (5592, 2944, 80, "down 256 128"), (4231, 1816, 80, "down 256 192"), (5699, 1448, 80, "down 256 224"),
    (4096, 2048, 1024, "both 256 192")])
def test_two_tile_widths(mok, T, H, I, widths):
    check(mok, T, H, I, "silu" if T % 2 else "gelu")


def test_dx_add(mok):
    for T, H, I in ((40, 136, 72), (900, 1032, 520)):  # tile kernel and pairs
        plan, d = check(mok, T, H, I, "silu", residual=False)
        w = (d["wg"], d["wu"], d["wd"])
        base = plan.grads.dx.double()
        add = torch.randn((T, H), device="cuda").to(BF)
        g = plan.backward(d["x"], *w, d["dy"], dx_add=add)
        # base was rounded once (2^-8 of it), the sum once more
        assert ((g.dx.double() - base - add.double()).abs() <= 2.0**-8 * (base.abs() + (base + add.double()).abs()) + 1e-6).all()
        want = g.dx.clone()
        plan.grads.dx.copy_(add)  # dx's own buffer
        assert torch.equal(plan.backward(d["x"], *w, d["dy"], dx_add=plan.grads.dx).dx, want)


def test_offsets_past_32_bits(mok):
    T, H, I = 270_000, 8192, 64  # x, out and the residual: 2.2 G values each
    x = torch.empty((T, H), dtype=BF, device="cuda").normal_()
    d = draw(1, H, I, 3)
    plan = mok.FFN(T, H, I, train=False)
    out = plan.forward(x, d["wg"], d["wu"], d["wd"], residual=x)
    for rows in (slice(0, 3), slice(T - 3, T)):
        t = [v.double() for v in (x[rows], d["wg"], d["wu"], d["wd"])]
        want, saved = ref.ffn(*t, "silu", t[0])
        near(out[rows], want, saved[4].abs() @ t[3].T.abs() + t[0].abs(), "out")
    assert plan.device_status() == 0


def test_wrong_layouts_are_refused(mok):
    d = draw(16, 64, 32, 2)
    plan = mok.FFN(16, 64, 32)
    for bad in (dict(x=d["x"].t().contiguous().t()), dict(wg=d["wg"].float()), dict(wd=d["wd"].t()), dict(x=d["x"][:8]),
                dict(x=d["x"].cpu())):
        a = {**d, **bad}
        with pytest.raises(ValueError):
            plan.forward(a["x"], a["wg"], a["wu"], a["wd"])
    buf = torch.empty(16 * 64 + 8, dtype=BF, device="cuda")
    with pytest.raises(mok.MokError):  # not 16-byte aligned
        plan.forward(buf[4:4 + 16 * 64].view(16, 64), d["wg"], d["wu"], d["wd"])
