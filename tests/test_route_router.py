"""The router's gradient on a schedule without the layer's staging: the tokens' width is the schedule's, and what does not go
with it is refused (without a GPU: before any device work)."""
import pytest
import torch

from test_gpu_route import gen

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def test_width_of_a_schedule(mok):
    assert mok.Routes(4, 8, 2, device="cpu").shape.H == 128
    r = mok.Routes(4, 8, 2, device="cpu", H=384)
    assert r.shape.H == 384 and r.rows == 4 * 2 + 8 * 127
    with pytest.raises(mok.MokError):
        mok.Routes(4, 8, 2, device="cpu", H=200)  # the router's widths are multiples of 128


@pytest.mark.parametrize("name,wrong", [("x", (4, 384)), ("w_router", (384, 8)), ("w_router", (256, 9)), ("dx", (4, 128)), ("dx", (5, 256))])
def test_sizes_that_are_not_the_schedules_are_refused(mok, name, wrong):
    routes = mok.Routes(4, 8, 2, device="cpu", H=256)
    sched = mok.Schedule(mok.mok_schedule(), routes.ws, None, None)
    sched.c.shape = routes.shape
    t = dict(x=torch.zeros((4, 256), dtype=BF), w_router=torch.zeros((256, 8), dtype=BF), dx=torch.zeros((4, 256), dtype=BF))
    t[name] = torch.zeros(wrong, dtype=BF)
    ids, w = torch.zeros((4, 2), dtype=I32), torch.zeros((4, 2))
    with pytest.raises(ValueError, match=rf"{name} must have the schedule's"):
        mok.router_backward(sched, t["x"], t["w_router"], ids, w, w, dx=t["dx"])


def test_a_gradient_that_is_not_the_schedules_is_refused(mok):
    sched = mok.Schedule(mok.mok_schedule(), None, None, None)
    sched.c.shape = mok.make_shape(4, 256, 128, 8, 2)
    x, wr, ids, w = torch.zeros((4, 256), dtype=BF), torch.zeros((256, 8), dtype=BF), torch.zeros((4, 2), dtype=I32), torch.zeros((4, 2))
    with pytest.raises(ValueError, match="dw_router must have the schedule's"):
        mok.mok_router_backward(sched, x, wr, ids, w, w, torch.zeros((128, 8)), None, x, False, torch.zeros(1 << 16, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,H", [(200, 8, 2, 256), (1, 16, 8, 512), (77, 5, 5, 128)])
def test_on_routes_as_on_the_layers_schedule(mok, T, E, K, H):
    """A step without the layer: router, routes, dispatch, combine, and back to the router's weights.  The gradients are
    equal to the ones on the layer's schedule."""
    _, n = gen(T + H)
    x, wr, dout = n(T, H).to(BF), (n(H, E) * 0.1).to(BF), n(T, H).to(BF)
    _, ids, w = mok.router_forward(x, wr, None, K)
    cfg, shape = mok.make_config(128, 256), mok.make_shape(T, H, 128, E, K)
    full = mok.mok_build_schedule(cfg, shape, ids, w, mok.alloc_workspace(cfg, shape))
    lean = mok.Routes(T, E, K, H=H).build(ids, w)
    rows = mok.dispatch(lean, x)
    _, d = mok.combine_backward(lean, rows, dout)
    got = mok.router_backward(lean, x, wr, ids, w, d, with_bias=True)
    want = mok.router_backward(full, x, wr, ids, w, d, with_bias=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.isfinite(got[0]).all()
    if H != 128:
        with pytest.raises(ValueError, match="x must have the schedule's"):
            mok.router_backward(mok.Routes(T, E, K).build(ids, w), x, wr, ids, w, d)
