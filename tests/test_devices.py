"""Which device a call of the binding runs on.  No GPU is needed: tensors "on" one are torch's fake tensors, which
have a device, a shape and a type but no memory."""
from unittest import mock

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from test_streams import _Streams

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


@pytest.mark.parametrize("stream", [None, 0x5550])
def test_ffn_backward_leaves_device_and_stream_to_x(mok, monkeypatch, stream):
    """As the forward: no stream given, none is chosen before x's device is known."""
    plan = mok.FFN(4, 64, 32, device="cpu")
    seen = {}

    class Bind:
        def __getattr__(self, name):
            return lambda *a: seen.update({name: a}) or ()
    monkeypatch.setattr(mok, "_bind", Bind())
    x, wg, wu, wd, dy, add = (torch.zeros(s, dtype=BF) for s in ((4, 64), (32, 64), (32, 64), (64, 32), (4, 64), (4, 64)))
    plan.forward(x, wg, wu, wd, stream=stream)
    assert seen["ffn_forward"][-1] == stream
    assert plan.backward(x, wg, wu, wd, dy, dx_add=add, stream=stream) is plan.grads
    got = seen["ffn_backward"]
    assert got[-1] == stream
    assert all(a is b for a, b in zip(got[-7:-1], (x, wg, wu, wd, dy, add)))


def test_ffn_backward_names_wrong_tensors(mok):
    plan = mok.FFN(4, 64, 32, device="cpu")
    with FakeTensorMode():
        make = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device="cuda:0")  # noqa: E731
        good = dict(x=make(4, 64), w_gate=make(32, 64), w_up=make(32, 64), w_down=make(64, 32), dy=make(4, 64))
        cases = [("x", make(5, 64)), ("w_gate", make(32, 64, dtype=F32)), ("w_up", make(64, 32)), ("w_down", None),
                 ("dy", make(4, 72)), ("dy", None), ("dx_add", make(4, 64, dtype=F32))]
    for name, bad in cases:
        with pytest.raises(ValueError, match=name):
            plan.backward(**{**good, name: bad})


def _tensors(device, **shapes):
    """{name: fake tensor}, each shape followed by the type.  (Where there are GPUs, torch would want this one.)"""
    with mock.patch.object(torch.cuda, "is_available", lambda: False), FakeTensorMode():
        return {k: torch.empty(s[:-1], dtype=s[-1], device=device) for k, s in shapes.items()}


def _dropout(mok, device):
    d = mok.Dropout.__new__(mok.Dropout)  # (its own checks want an address)
    d.rng = _tensors(device, rng=(2, torch.int64))["rng"]
    d._placed = mok._placed_dropout(mok.mok_dropout(0.1, 0x1000), d.rng.device.index)
    d.addr = mok.ctypes.addressof(d._placed)
    return d


CALLS = {
    "rmsnorm_forward": (dict(x=(4, 64, BF), weight=(64, BF), residual=(4, 64, F32)), dict(eps=1e-6)),
    "rmsnorm_backward": (dict(h=(4, 64, F32), rstd=(4, F32), weight=(64, BF), dy=(4, 64, BF), dres=(4, 64, F32)), {}),
    "dropout_forward": (dict(x=(4, 64, BF), residual=(4, 64, F32), out=(4, 64, F32)), {}),
    "dropout_backward": (dict(dout=(4, 64, F32), dx=(4, 64, BF)), {}),
}
ELSEWHERE = [(c, k) for c, (t, _) in CALLS.items() for k in (*list(t)[1:], "dropout.rng")]


@pytest.mark.parametrize("call,name", ELSEWHERE)
def test_operands_on_another_device_are_refused(mok, call, name):
    tensors, other = CALLS[call]
    a = _tensors("cuda:0", **tensors)
    if name in a:
        a[name] = _tensors("cuda:1", **{name: tensors[name]})[name]
    drop = _dropout(mok, "cuda:1" if name == "dropout.rng" else "cuda:0")
    with pytest.raises(ValueError, match=f"{name} must be on cuda:0.*got cuda:1"):
        getattr(mok, call)(**a, **other, dropout=drop)


FFN = dict(x=(4, 64, BF), w_gate=(32, 64, BF), w_up=(32, 64, BF), w_down=(64, 32, BF))


@pytest.mark.parametrize("call,name", [("forward", k) for k in ("w_gate", "w_up", "w_down", "residual", "the plan")] +
                         [("backward", k) for k in ("w_gate", "w_up", "w_down", "dy", "dx_add", "the plan")])
def test_ffn_operands_on_another_device_are_refused(mok, call, name):
    plan = mok.FFN(4, 64, 32, device="cpu")
    plan.out = _tensors("cuda:1" if name == "the plan" else "cuda:0", out=(4, 64, BF))["out"]
    place = plan.out.device.index
    plan._fwd, plan._bwd = (place, *plan._fwd[1:]), (place, *plan._bwd[1:])
    shapes = {**FFN, **(dict(residual=(4, 64, BF)) if call == "forward" else dict(dy=(4, 64, BF), dx_add=(4, 64, BF)))}
    a = _tensors("cuda:0", **shapes)
    if name in a:
        a[name] = _tensors("cuda:1", **{name: shapes[name]})[name]
    with pytest.raises(ValueError, match=f"{name} must be on cuda:0.*got cuda:1"):
        getattr(plan, call)(**a)


def test_sublayer_refuses_other_devices_before_it_runs(mok):
    from mixture_experts_layer_build_gb300.sublayer import Params, Sublayer
    T, H, I, E, K, Is = 4, 128, 128, 4, 2, 32
    sub = Sublayer(T, H, I, E, K, Is, device="cpu")
    shapes = dict(w_norm=(H, BF), w_router=(H, E, BF), w_gate=(E, I, H, BF), w_up=(E, I, H, BF), w_down=(E, H, I, BF),
                  s_gate=(Is, H, BF), s_up=(Is, H, BF), s_down=(H, Is, BF))
    here = {k: torch.empty(s[:-1], dtype=s[-1]) for k, s in shapes.items()}
    x = torch.empty((T, H), dtype=BF)
    away = _tensors("cuda:0", x=(T, H, BF), **shapes)
    for call, name in ((sub.forward, "branch"), (sub.backward, "dout")):
        with pytest.raises(ValueError, match=f"{name} must be on cpu.*got cuda:0"):
            call(away["x"], x, Params(**here))
        with pytest.raises(ValueError, match="s_up must be on cpu.*got cuda:0"):
            call(x, x, Params(**{**here, "s_up": away["s_up"]}))


def test_streams_of_another_device_are_refused(mok, monkeypatch):
    streams = _Streams(monkeypatch)
    a = _tensors("cuda:0", x=(4, 64, BF), w=(64, BF), g=(32, 64, BF), d=(64, 32, BF))
    x, drop, s = a["x"], _dropout(mok, "cuda:0"), streams.Stream(0x5550, 1)
    plan = mok.FFN(4, 64, 32, device="cpu")
    for call in (lambda: mok.rmsnorm_forward(x, a["w"], 1e-6, stream=s), lambda: mok.dropout_forward(x, drop, stream=s),
                 lambda: mok.rmsnorm_backward(x, a["w"], a["w"], x, stream=s),
                 lambda: mok.dropout_backward(x, drop, stream=s),
                 lambda: plan.forward(x, a["g"], a["g"], a["d"], stream=s),
                 lambda: plan.backward(x, a["g"], a["g"], a["d"], x, stream=s)):
        with pytest.raises(ValueError, match="stream must be on cuda:0.*got cuda:1"):
            call()


def test_a_handle_is_of_the_tensors_device(mok, monkeypatch):
    streams = _Streams(monkeypatch)
    x = _tensors("cuda:1", x=(4, 64, BF))["x"]
    for handle in (0, 0x5550):
        with mok._on_stream(handle, x):
            assert [(s.cuda_stream, s.device.index) for s in streams.current] == [(handle, 1)]
