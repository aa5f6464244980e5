"""Which device a call of the binding runs on.  No GPU is needed: tensors "on" one are torch's fake tensors, which
have a device, a shape and a type but no memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

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
