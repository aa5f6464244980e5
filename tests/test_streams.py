"""The stream that a call of the binding is given: which stream it runs on, and which one owns what it allocates.

Without a GPU torch's stream objects are stood in for; on one, the allocator's own record of each block's owner is
read."""
import contextlib

import pytest
import torch

BF = torch.bfloat16


@pytest.fixture(scope="module")
def mok():
    import __graft_entry__
    __graft_entry__.build_library()
    from mixture_experts_layer_build_gb300 import mok as m
    return m


class _Streams:
    """torch.cuda's stream functions on stand-ins; `current` is the stack of streams made current."""

    class Stream:
        def __init__(self, handle, device=0):
            self.cuda_stream, self.device = handle, torch.device("cuda", device)

    def __init__(self, monkeypatch):
        self.current, pool = [], iter(range(0x7000, 0x8000, 16))
        index = lambda d: 0 if d is None else torch.device(d).index or 0  # noqa: E731
        for name, f in dict(
                Stream=self.Stream,
                # a handle of 0 gives a new stream, as torch's own class does
                ExternalStream=lambda h, device=None: self.Stream(h or next(pool), index(device)),
                default_stream=lambda device=None: self.Stream(0, index(device)),
                stream=self._stream).items():
            monkeypatch.setattr(torch.cuda, name, f)

    @contextlib.contextmanager
    def _stream(self, s):
        self.current.append(s)
        yield
        self.current.pop()


@pytest.mark.parametrize("handle", [0, 0x5550])
def test_a_handle_stands_for_its_own_stream(mok, monkeypatch, handle):
    streams = _Streams(monkeypatch)
    with mok._on_stream(handle):
        assert [s.cuda_stream for s in streams.current] == [handle]


class _Recorder:
    """Stands in for a library call, and notes the stream that is current at it and at each torch.empty before it."""

    def __init__(self, monkeypatch, streams, module, name):
        self.at = []
        note = lambda: self.at.append(streams.current[-1].cuda_stream if streams.current else None)  # noqa: E731
        empty = torch.empty

        def allocate(*a, **k):
            note()
            return empty(*a, **k)
        monkeypatch.setattr(torch, "empty", allocate)
        monkeypatch.setattr(module, name, lambda *a, **k: note())


def test_router_allocates_on_the_stream_it_runs_on(mok, monkeypatch):
    streams = _Streams(monkeypatch)
    x, w = torch.zeros((4, 128), dtype=BF), torch.zeros((128, 8), dtype=BF)
    calls = _Recorder(monkeypatch, streams, mok, "mok_router_forward")
    mok.router_forward(x, w, None, 2, stream=0x5550)
    assert calls.at == [0x5550] * 4  # logits, ids, weights, the call
    ids, s = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    sched = mok.Schedule(mok.mok_schedule(), None, ids, s)
    sched.c.shape = mok.make_shape(4, 128, 128, 8, 2)
    calls = _Recorder(monkeypatch, streams, mok, "mok_router_backward")
    mok.router_backward(sched, x, w, ids, s, s, with_bias=True, stream=0x5550)
    assert calls.at[-4:] == [0x5550] * 4  # dw, db, ws, the call


def test_weight_copies_are_made_on_the_given_stream(mok, monkeypatch):
    """Allocations and transposes of quantize_weights: a transposed copy is read by the kernel of the given stream and
    dropped at once."""
    streams = _Streams(monkeypatch)
    at = []
    note = lambda: at.append(streams.current[-1].cuda_stream if streams.current else None)  # noqa: E731
    contiguous = torch.Tensor.contiguous
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: (note(), contiguous(t))[1])
    monkeypatch.setattr(mok._lib, "mok_mxfp8_quantize", lambda *a: note() or 0)
    monkeypatch.setattr(mok, "_ptr", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(mok, "_stream", lambda s: 0 if s is None else int(s))
    w = torch.zeros((2, 64, 64), dtype=BF)
    assert set(mok.quantize_weights(w, w, w, stream=0x5550)) == set(mok.MX_KEYS)
    assert at == [0x5550] * 9  # six calls, three transposes
    at.clear()
    calls = _Recorder(monkeypatch, streams, mok._lib, "mok_mxfp8_quantize")
    monkeypatch.setattr(mok, "_check", lambda rc, where: None)
    mok.mok_mxfp8_quantize(w[0], stream=0x5550)
    assert calls.at == [0x5550] * 3  # codes, scales, the call


def owner(t):
    """Handle of the stream that owns t's memory, by the allocator's record."""
    return next(p["stream"] for p in torch.cuda.memory_snapshot()
                if p["address"] <= t.data_ptr() < p["address"] + p["total_size"])


@pytest.mark.gpu
def test_handle_of_the_default_stream(mok):
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((200, 512), generator=g).to(BF).cuda(), torch.ones(512, dtype=BF, device="cuda")
    want = mok.rmsnorm_forward(x, w, 1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = mok.rmsnorm_forward(x, w, 1e-6, stream=torch.cuda.default_stream().cuda_stream)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert owner(o.y) == 0 and owner(o.rstd) == 0
    assert torch.equal(o.y, want.y) and torch.equal(o.rstd, want.rstd)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_sublayer_on_a_given_stream(mok, handle):
    """Forward and backward of a sublayer on a stream that is not the current one: results as on the current stream, and
    every tensor of the router and the norm owned by that stream."""
    from mixture_experts_layer_build_gb300.sublayer import Params, Sublayer
    T, H, I, E, K, Is = 300, 256, 128, 8, 2, 200
    g = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    p = Params(**{k: (n(*s) * 1.5 / H**0.5).to(BF).cuda() for k, s in dict(
        w_norm=(H,), w_router=(H, E), w_gate=(E, I, H), w_up=(E, I, H), w_down=(E, H, I), s_gate=(Is, H), s_up=(Is, H),
        s_down=(H, Is)).items()})
    branch, dout, res, dh = n(T, H).to(BF).cuda(), n(T, H).to(BF).cuda(), n(T, H).cuda(), n(T, H).cuda()
    drop = mok.Dropout(0.1, torch.tensor([3, 4], device="cuda"))

    def step(sub, stream):
        out, h = sub.forward(branch, res, p, drop, stream=stream)
        dbranch, dres, grads = sub.backward(dout, dh, p, drop, stream=stream)
        return [out, h, dbranch, dres, *vars(grads).values()], grads
    want, _ = step(Sublayer(T, H, I, E, K, Is), None)
    sub = Sublayer(T, H, I, E, K, Is)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, grads = step(sub, side.cuda_stream if handle else side)
    assert torch.cuda.current_stream() != side
    for t in (sub.norm.h, sub.norm.y, sub.norm.rstd, sub.ids, sub.weights, grads.w_router, grads.w_norm, got[2], got[3]):
        assert owner(t) == side.cuda_stream
    torch.cuda.synchronize()
    assert sub.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_weight_copies_on_a_given_stream(mok):
    g = torch.Generator().manual_seed(6)
    w = [torch.randn(s, generator=g).to(BF).cuda() for s in ((3, 128, 256), (3, 128, 256), (3, 256, 128))]
    want = mok.quantize_weights(*w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mok.quantize_weights(*w, stream=side)
    assert all(owner(t) == side.cuda_stream for t in got.values())
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.gpu
def test_device_status_waits_for_every_stream(mok):
    from mixture_experts_layer_build_gb300.sublayer import Sublayer
    sub = Sublayer(16, 128, 128, 4, 2, 64)
    ids, w = torch.zeros((16, 2), dtype=torch.int32, device="cuda"), torch.ones((16, 2), device="cuda")
    ids[:, 1] = 1
    side = torch.cuda.Stream()

    def later(read):  # a problem that a kernel on another stream finds in half a second
        sub.ffn.status.zero_()
        sub.layer.schedule(ids, w)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(1_000_000_000)
            sub.ffn.status.fill_(1 << mok.MOK_ERR_TIMEOUT)
            sub.layer.sched._view("status", 1).fill_(1 << mok.MOK_ERR_BAD_EXPERT_ID)
        return read()
    assert later(sub.ffn.device_status) == 1 << mok.MOK_ERR_TIMEOUT
    assert later(sub.device_status) == 1 << mok.MOK_ERR_TIMEOUT | 1 << mok.MOK_ERR_BAD_EXPERT_ID
