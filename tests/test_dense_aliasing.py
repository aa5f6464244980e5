"""Buffers of the feed-forward backward that may not overlap: dx is written by the launch that reads x and dy for the
weight gradients.  Refused on the host, so fake addresses never reach a device."""
import ctypes

import pytest

A = 0x100000  # a 256-byte aligned address that nothing reads


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


T, H, I = 4, 64, 32
BYTES = T * H * 2


@pytest.mark.parametrize("which", ["x", "dy"])
@pytest.mark.parametrize("off", [0, 16, -16, BYTES - 16, 16 - BYTES])
def test_dx_over_an_input_of_the_weight_gradients_is_refused(mok, which, off):
    place = dict(x=A + 0x10000, dy=A + 0x20000)
    dx = place[which] + off
    grads = mok.mok_ffn_grads(dx, *((A, A, None) if which == "x" else (None, None, A)), 0)
    rc = mok._lib.mok_ffn_backward(ctypes.byref(mok.mok_ffn_shape(T, H, I, 0)), place["x"], A, A, A, A, 1 << 30,
                                   place["dy"], ctypes.byref(grads), A, 1 << 30, None, None)
    assert rc == mok.MOK_ERR_INVALID_ARG


def test_a_plans_own_dx_is_named(mok, monkeypatch):
    import torch
    plan = mok.FFN(T, H, I, device="cpu")
    x, g, d = (torch.zeros(s, dtype=torch.bfloat16) for s in ((T, H), (I, H), (H, I)))

    class Bind:  # the library's answer for a buffer that overlaps
        def ffn_backward(self, *a):
            return mok.MOK_ERR_INVALID_ARG
    monkeypatch.setattr(mok, "_bind", Bind())
    with pytest.raises(ValueError, match="dy must not be the plan's dx"):
        plan.backward(x, g, g, d, plan.grads.dx)
    with pytest.raises(ValueError, match="x must not be the plan's dx"):
        plan.backward(plan.grads.dx, g, g, d, x)
    with pytest.raises(mok.MokError):
        plan.backward(x, g, g, d, x)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(40, 136, 72), (900, 1032, 520)])  # tile kernel and pairs
def test_dx_in_the_buffer_of_an_input_that_nothing_else_reads(mok, T, H, I):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    x, wg, wu, wd, dy = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                         for s in ((T, H), (I, H), (I, H), (H, I), (T, H)))
    plan = mok.FFN(T, H, I)
    plan.forward(x, wg, wu, wd)
    want = plan.backward(x, wg, wu, wd, dy)
    over_dy, over_x = dy.clone(), x.clone()
    dw = {k: torch.zeros_like(getattr(want, k)) for k in ("dw_gate", "dw_up", "dw_down")}
    for at, x_, dy_, keep in ((over_dy, x, over_dy, ("dw_gate", "dw_up")), (over_x, over_x, dy, ("dw_down",))):
        grads = mok.mok_ffn_grads(at.data_ptr(), *(t.data_ptr() if k in keep else None for k, t in dw.items()), 0)
        rc = mok._lib.mok_ffn_backward(ctypes.byref(plan.shape), x_.data_ptr(), wg.data_ptr(), wu.data_ptr(), wd.data_ptr(),
                                       plan.ctx.data_ptr(), plan.ctx.numel(), dy_.data_ptr(), ctypes.byref(grads),
                                       plan.ws.data_ptr(), plan.ws.numel(), None, mok._stream(None))
        assert rc == mok.MOK_OK
    assert torch.equal(over_dy, want.dx) and torch.equal(over_x, want.dx)
    assert all(torch.equal(t, getattr(want, k)) for k, t in dw.items())
    with pytest.raises(ValueError, match="dy must not be the plan's dx"):
        plan.backward(x, wg, wu, wd, plan.grads.dx)
