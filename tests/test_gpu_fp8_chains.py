"""Calls right behind one another through buffers that are used again: a kernel that starts early reads what the one in front
has written, and does not write what that one still reads.  The same steps with a wait after each call are the reference, bit for bit."""
import pytest
import torch

from test_gpu_fp8 import codes
from test_gpu_route import gen, routing

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def captured(f):
    """f in a graph, after a run of it on a side stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    return graph


@pytest.mark.parametrize("M", [1, 5, 8, 9, 40, 200])
def test_chained_linears(mok, M):
    """Each linear's output is the next one's input, in two buffers that change places, and its own copy is kept: few rows (read
    by the product itself), some, and pairs."""
    W, steps = 1032, 40
    _, n = gen(M)
    ws = [mok.fp8_quantize_weight((n(W, W) * W**-0.5).to(BF))[0] for _ in range(4)]
    a, b, x = (n(M, W).to(BF) for _ in range(3))
    kept = torch.empty((steps, M, W), dtype=BF, device="cuda")

    def run(wait):
        a.copy_(x)
        for i in range(steps):
            src, dst = (a, b) if i % 2 == 0 else (b, a)
            mok.fp8_linear(src, ws[i % 4], out=dst)
            if wait:
                torch.cuda.synchronize()
            mok.fp8_linear(dst, ws[(i + 1) % 4], out=kept[i])  # read again by another call
            if wait:
                torch.cuda.synchronize()
    graph = captured(lambda: run(False))
    for k in range(4):
        x.copy_(n(M, W))
        run(True)
        want = kept.clone()
        assert torch.isfinite(want.float()).all()
        kept.zero_()
        run(False)
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


@pytest.mark.parametrize("T,E,K", [(1, 16, 4), (20, 8, 2), (400, 6, 2)])
def test_chained_expert_blocks(mok, T, E, K):
    """Dispatch, up, quantise, down, combine, again and again over the same rows, with a routing of each step's own."""
    H, I, steps = 264, 392, 12
    _, n = gen(T)
    up, down = codes(I, H, 1, block=True, batch=E, mok=mok), codes(H, I, 2, block=True, batch=E, mok=mok)
    up.s.mul_(1e-3), down.s.mul_(1e-3)
    routings = [routing("spread", T, E, K, seed=i) for i in range(steps)]
    routes = mok.Routes(T, E, K)
    hid = torch.zeros((routes.rows, I), dtype=BF, device="cuda")
    y = torch.zeros((routes.rows, H), dtype=BF, device="cuda")
    x, h = n(T, H).to(BF), torch.empty((T, H), dtype=BF, device="cuda")
    kept = torch.empty((steps, T, H), dtype=BF, device="cuda")

    def run(wait):
        sync = torch.cuda.synchronize if wait else lambda: None
        h.copy_(x)
        for i in range(steps):
            s = routes.build(*routings[i])
            sync()
            a, _ = mok.dispatch_fp8(s, h)
            sync()
            mok.fp8_grouped_matmul(s, a, up, out=hid)
            sync()
            b, _ = mok.fp8_quantize(hid, sched=s)
            sync()
            mok.fp8_grouped_matmul(s, b, down, out=y)
            sync()
            mok.combine(s, y, out=h)
            sync()
            mok.combine(s, y, out=kept[i])
            sync()
    graph = captured(lambda: run(False))
    for k in range(4):
        x.copy_(n(T, H))
        run(True)
        want = kept.clone()
        assert torch.isfinite(want.float()).all() and (want[-1] != 0).any()
        for again in (lambda: run(False), graph.replay):
            kept.zero_()
            again()
            torch.cuda.synchronize()
            assert torch.equal(kept, want)
