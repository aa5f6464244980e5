"""Copies of the objects that keep addresses for the library: each has to have its own.  No GPU needed."""
import copy
import pickle

import pytest
import torch

COPIES = [copy.copy, copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))]


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


@pytest.mark.parametrize("make", COPIES)
@pytest.mark.parametrize("train", [False, True])
def test_a_copied_plan_has_its_own_buffers(mok, make, train):
    plan = mok.FFN(16, 64, 32, act="gelu", train=train, dw_dtype=torch.float32, device="cpu")
    twin = make(plan)
    buffers = ["out", "ctx", "status"] + (["ws"] if train else [])
    for k in buffers:
        a, b = getattr(plan, k), getattr(twin, k)
        assert a.shape == b.shape and a.dtype == b.dtype and a.data_ptr() != b.data_ptr(), k
    for k in ("out", "ctx", "status"):
        assert getattr(twin, k).data_ptr() in twin._fwd and getattr(plan, k).data_ptr() not in twin._fwd, k
    assert mok.ctypes.addressof(twin.shape) in twin._fwd and mok.ctypes.addressof(plan.shape) not in twin._fwd
    assert (twin.T, twin.H, twin.I, twin.shape.act, twin.train) == (16, 64, 32, plan.shape.act, train)
    if train:
        assert twin.ws.data_ptr() in twin._bwd and mok.ctypes.addressof(twin._grads) in twin._bwd
        assert twin.grads.dw_gate.dtype == torch.float32
        assert twin._grads.dw_down == twin.grads.dw_down.data_ptr() != plan.grads.dw_down.data_ptr()


@pytest.mark.parametrize("make", COPIES)
def test_a_copied_dropout_points_at_its_own_state(mok, make, monkeypatch):
    monkeypatch.setattr(mok, "_ptr", lambda t, *a: t.data_ptr())  # (a state on the CPU)
    arg = mok._arg
    monkeypatch.setattr(mok, "_arg", lambda t, *a: t.data_ptr() if not t.is_cuda else arg(t, *a))
    index = mok._placed_dropout
    monkeypatch.setattr(mok, "_placed_dropout", lambda d, i: index(d, -1 if i is None else i))
    drop = mok.Dropout(0.25, torch.tensor([7, 9]))
    twin = make(drop)
    assert twin.c.p == 0.25 and torch.equal(twin.rng, drop.rng)
    assert twin.c.rng == twin.rng.data_ptr() and twin.addr == mok.ctypes.addressof(twin._placed) != drop.addr
