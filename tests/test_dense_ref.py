"""The dense operators' 64-bit references (tests/dense_ref.py) against published values, autograd and
central differences, and the host-side refusals of their entry points (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import dense_ref as ref


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


# known-answer vectors of Philox4x32-10 published with the generator: counter, key -> output
KAT = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
       ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
       ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
        (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]


@pytest.mark.parametrize("counter,key,want", KAT)
def test_generator_matches_its_published_vectors(counter, key, want):
    assert tuple(ref.philox4x32_10(counter, key)) == want


def test_draws_are_the_words_halves_in_memory_order():
    seed, offset, first = 0x0123456789ABCDEF, 0xFEDCBA9876543210, (1 << 32) - 1  # crosses a counter word
    d = ref.draws16(24, seed, offset, first)
    for i in range(3):
        g = first + i
        w = ref.philox4x32_10((g & 0xFFFFFFFF, g >> 32, offset & 0xFFFFFFFF, offset >> 32),
                              (seed & 0xFFFFFFFF, seed >> 32))
        assert d[8 * i:8 * i + 8].tolist() == [v for x in w for v in (x & 0xFFFF, x >> 16)]


def test_dropout_threshold_and_share():
    assert [ref.threshold(p) for p in (0.0, 0.5, 1.0, 1e-6)] == [0, 32768, 65536, 0]
    kept = ref.keep((400, 1000), 0.1, 7, 3).double().mean().item()
    assert abs(kept - 0.9) < 5 * (0.09 / 400000) ** 0.5


def _leaf(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64).requires_grad_()


def test_norm_gradient_formula():
    g = torch.Generator().manual_seed(0)
    h, w = _leaf(g, 5, 24), _leaf(g, 24)
    dy = torch.randn((5, 24), generator=g, dtype=torch.float64)
    y, rstd = ref.rmsnorm(h, w, 1e-6)
    y.backward(dy)
    dh, dw = ref.rmsnorm_grads(h.detach(), rstd.detach(), w.detach(), dy, None)
    assert torch.allclose(dh, h.grad, rtol=1e-12, atol=1e-13) and torch.allclose(dw, w.grad, rtol=1e-12, atol=1e-13)
    e = 1e-6  # central differences of <y, dy> along a direction
    d = torch.randn((5, 24), generator=g, dtype=torch.float64)
    f = lambda s: (ref.rmsnorm(h.detach() + s * d, w.detach(), 1e-6)[0] * dy).sum()  # noqa: E731
    assert abs(((f(e) - f(-e)) / (2 * e) - (dh * d).sum()).item()) < 1e-7


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_ffn_gradient_formula(kind):
    g = torch.Generator().manual_seed(1)
    x, wg, wu, wd = _leaf(g, 4, 16), _leaf(g, 24, 16), _leaf(g, 24, 16), _leaf(g, 16, 24)
    dy = torch.randn((4, 16), generator=g, dtype=torch.float64)
    out, saved = ref.ffn(x, wg, wu, wd, kind)
    out.backward(dy)
    t = [v.detach() for v in (x, wg, wu, wd)]
    got, _ = ref.ffn_grads(*t, dy, ref.ffn(*t, kind)[1])
    for k, leaf in (("dx", x), ("dw_gate", wg), ("dw_up", wu), ("dw_down", wd)):
        assert torch.allclose(got[k], leaf.grad, rtol=1e-11, atol=1e-11), k
    e = 1e-6
    d = torch.randn((24, 16), generator=g, dtype=torch.float64)
    f = lambda s: (ref.ffn(t[0], t[1] + s * d, t[2], t[3], kind)[0] * dy).sum()  # noqa: E731
    num = ((f(e) - f(-e)) / (2 * e)).item()
    assert abs(num - (got["dw_gate"] * d).sum().item()) < 1e-6 * max(1.0, abs(num))
    want = torch.nn.functional.silu(x) if kind == "silu" else torch.nn.functional.gelu(x, approximate="tanh")
    assert torch.allclose(ref.act(x, kind)[0], want, rtol=1e-12, atol=1e-13)


# ---- host-side refusals: nothing is enqueued, so fake addresses never reach a device ----
A = 0x10000  # a 256-byte aligned address that nothing reads


def _drop(mok, p=0.1, rng=A):
    return ctypes.byref(mok.mok_dropout(p, rng))


def test_dropout_refusals(mok):
    f, b = mok._lib.mok_dropout_forward, mok._lib.mok_dropout_backward
    bad = mok.MOK_ERR_INVALID_ARG
    assert f(0, 0, _drop(mok), None, None, None, None) == mok.MOK_OK
    assert f(8, 0, None, A, A, A, None) == bad
    for n in (-8, 4, 12):
        assert f(n, 0, _drop(mok), A, A, A, None) == bad
        assert b(n, 0, _drop(mok), A, A, None) == bad
    for d in (_drop(mok, -0.1), _drop(mok, 1.1), _drop(mok, float("nan")), _drop(mok, 0.1, None), _drop(mok, 0.1, A + 4)):
        assert f(8, 0, d, A, A, A, None) == bad
        assert b(8, 0, d, A, A, None) == bad
    assert f(8, 2, _drop(mok), A, A, A, None) == bad
    for args in ((None, A, A), (A + 2, A, A), (A, A + 8, A), (A, A, None), (A, A, A + 8)):
        assert f(8, 0, _drop(mok), *args, None) == bad


def test_norm_refusals(mok):
    f = mok._lib.mok_rmsnorm_forward
    bad = mok.MOK_ERR_INVALID_ARG

    def fwd(T=4, H=64, st=0, eps=1e-6, x=A, res=A, drop=None, w=A, h=A, y=A, q=None, s=None, rstd=A):
        return f(ctypes.byref(mok.mok_norm_shape(T, H, st, eps)), x, res, drop, w, h, y, q, s, rstd, None)

    assert fwd(T=0) == mok.MOK_OK
    for kw in (dict(T=-1), dict(H=0), dict(H=12), dict(H=16392), dict(st=3), dict(eps=-1.0), dict(eps=float("inf")),
               dict(eps=float("nan")), dict(x=None), dict(w=None), dict(y=None), dict(q=A), dict(s=A), dict(h=None),
               dict(h=None, res=None, st=1), dict(h=None, res=None, drop=_drop(mok)), dict(x=A + 8), dict(y=A + 4),
               dict(rstd=A + 2), dict(H=40, q=A, s=A), dict(drop=_drop(mok, 2.0))):
        assert fwd(**kw) == bad, kw
    assert f(None, A, A, None, A, A, A, None, None, A, None) == bad

    def wsb(T, H):
        return mok._lib.mok_rmsnorm_workspace_bytes(ctypes.byref(mok.mok_norm_shape(T, H, 0, 0.0)))
    assert wsb(4, 12) == 0 and wsb(0, 64) == 256 and wsb(100000, 4096) % 256 == 0
    b = mok._lib.mok_rmsnorm_backward

    def bwd(T=4, H=64, h=A, rstd=A, w=A, dy=A, dres=None, dh=A, dx=None, dw=A, ws=A, n=1 << 30):
        return b(ctypes.byref(mok.mok_norm_shape(T, H, 0, 0.0)), h, rstd, w, dy, dres, None, dh, dx, dw, ws, n, None)
    for kw in (dict(H=20), dict(h=None), dict(rstd=None), dict(w=None), dict(dy=None), dict(dw=None), dict(ws=None),
               dict(ws=A + 16), dict(dres=A + 8), dict(dh=A + 8), dict(dx=A + 2), dict(rstd=A + 1)):
        assert bwd(**kw) == bad, kw
    assert bwd(n=16) == mok.MOK_ERR_WORKSPACE_TOO_SMALL


def test_ffn_refusals(mok):
    bad, small = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_WORKSPACE_TOO_SMALL

    def shape(T=4, H=64, I=32, act=0):
        return ctypes.byref(mok.mok_ffn_shape(T, H, I, act))
    for kw in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=20), dict(I=12), dict(H=65544), dict(I=-8), dict(act=2)):
        assert mok._lib.mok_ffn_ctx_bytes(shape(**kw), 1) == 0, kw
        assert mok._lib.mok_ffn_workspace_bytes(shape(**kw)) == 0, kw
    n0, n1 = (mok._lib.mok_ffn_ctx_bytes(shape(T=1000, I=1000), s) for s in (0, 1))
    assert n0 >= 2 * 1000 * 1000 and n1 >= 10 * 1000 * 1000 and n0 % 256 == 0 and n1 % 256 == 0
    f = mok._lib.mok_ffn_forward

    def fwd(sh=None, x=A, wg=A, wu=A, wd=A, res=None, out=A, ctx=A, n=1 << 30, save=1, status=None):
        return f(sh or shape(), x, wg, wu, wd, res, out, ctx, n, save, status, None)
    assert fwd(shape(T=0), x=None, out=None) == mok.MOK_OK
    for kw in (dict(x=None), dict(wg=None), dict(wu=A + 8), dict(wd=None), dict(res=A + 8), dict(out=None),
               dict(ctx=None), dict(ctx=A + 16), dict(status=A + 2), dict(sh=shape(H=20))):
        assert fwd(**kw) == bad, kw
    assert fwd(n=64) == small
    b = mok._lib.mok_ffn_backward

    def bwd(g=(A, A, A, A, 0), x=A, ctx=A, n=1 << 30, dy=A, ws=A, wn=1 << 30, grads=True):
        gr = mok.mok_ffn_grads(*g)
        return b(shape(), x, A, A, A, ctx, n, dy, ctypes.byref(gr) if grads else None, ws, wn, None, None)
    for kw in (dict(grads=False), dict(g=(A, A, None, A, 0)), dict(g=(A, A, A, A, 2)), dict(g=(A + 2, A, A, A, 0)),
               dict(g=(A, A, A, A + 8, 0)), dict(x=None), dict(dy=None), dict(ctx=None), dict(ws=None), dict(ws=A + 8)):
        assert bwd(**kw) == bad, kw
    assert bwd(n=64) == small and bwd(wn=64) == small


def test_binding_refuses_wrong_tensors(mok):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        mok.rmsnorm_forward(x, torch.zeros(64, dtype=torch.bfloat16), 1e-6)
    with pytest.raises(ValueError):
        mok.Dropout(0.1, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        mok.FFN(4, 64, 32, act="tanh", device="cpu")
    with pytest.raises(mok.MokError):
        mok.FFN(4, 60, 32, device="cpu")
    plan = mok.FFN(4, 64, 32, train=False, device="cpu")
    with pytest.raises(ValueError):
        plan.backward(x, x, x, x, x)
    with pytest.raises(ValueError):
        plan.forward(torch.zeros((5, 64), dtype=torch.bfloat16), x, x, x)
    assert np.prod(plan.ctx.shape) == mok.mok_ffn_ctx_bytes(plan.shape, False)
