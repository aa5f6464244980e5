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
