"""What the quantising calls return is memory of its own, tensor by tensor: to be saved, kept in part, or used on another stream."""
import io

import pytest
import torch

import fp8_ref as ref
from test_gpu_route import gen, routing

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def mok():
    from mixture_experts_layer_build_gb300 import mok as m
    return m


def made(mok):
    """{name: Fp8} of every quantising call, with sizes that fill no block."""
    _, n = gen(2)
    x, w, we = n(150, 264).to(BF), n(136, 264).to(BF), n(3, 136, 264).to(BF)
    sched = mok.Routes(150, 3, 2).build(*routing("spread", 150, 3, 2))
    return {f"{k} {i}": m for k, pair in dict(
        rows=mok.fp8_quantize(x, transposed=True), weight=mok.fp8_quantize_weight(w, transposed=True),
        weights=mok.fp8_quantize_weight(we, transposed=True), dispatch=mok.dispatch_fp8(sched, x, transposed=True),
        routed=mok.fp8_quantize(n(sched.c.rpad_max, 136).to(BF), transposed=True, sched=sched)).items() for i, m in enumerate(pair)}


def test_saved_and_loaded(mok):
    got = made(mok)
    for part in [{k: dict(q=m.q, s=m.s) for k, m in got.items()}, {"one": dict(q=got["weights 0"].q, s=got["weights 0"].s)}]:
        f = io.BytesIO()
        torch.save(part, f)
        f.seek(0)
        back = torch.load(f)
        for k, m in part.items():
            assert torch.equal(back[k]["q"], m["q"]) and torch.equal(back[k]["s"].view(torch.int32), m["s"].view(torch.int32))
    lw, w = made(mok)["weight 0"], torch.load(_saved(dict(q=got["weight 0"].q, s=got["weight 0"].s)))
    x = gen(3)[1](40, 264).to(BF)
    assert torch.equal(mok.fp8_linear(x, mok.Fp8(w["q"], w["s"], 264, True)), mok.fp8_linear(x, lw))


def _saved(d):
    f = io.BytesIO()
    torch.save(d, f)
    f.seek(0)
    return f


def test_every_tensor_has_a_storage_of_its_own(mok):
    seen = set()
    got = made(mok)
    for k, m in got.items():
        for t in (m.q, m.s):
            at, size, own = t.untyped_storage().data_ptr(), t.untyped_storage().nbytes(), t.data_ptr()
            assert at == own and size == t.numel() * t.element_size() and at % 256 == 0 and at not in seen, k
            seen.add(at)
            assert t.is_contiguous() and t.storage_offset() == 0 and not t.requires_grad and t.device == torch.device("cuda", 0), k


def test_scales_outlive_their_codes(mok):
    """The codes' memory goes back to the allocator when they are dropped; the scales stay, and the other way round."""
    x = gen(4)[1](8192, 4096).to(BF)
    want_q, want_s = ref.quantize(x, (1, 128))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    m, _ = mok.fp8_quantize(x)
    s = m.s
    del m
    held = torch.cuda.memory_allocated() - before
    assert held < 8192 * 4096 // 4  # 1 MB of scales, in a block of up to twice that
    junk = torch.full((8192 * 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(s.T.double(), want_s)
    del junk, s
    q = mok.fp8_quantize(x)[0].q
    assert torch.equal(ref.decode(q), want_q)


def test_used_on_another_stream(mok):
    """record_stream on the scales alone holds their memory back until that stream's work has ended."""
    x = gen(5)[1](2048, 2048).to(BF)
    side = torch.cuda.Stream()
    m, _ = mok.fp8_quantize(x)
    want = m.s.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        kept = m.s + 0
    m.s.record_stream(side)
    at, size = m.s.data_ptr(), m.s.shape
    del m
    others = [torch.zeros(size, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() != at for t in others)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_where_torch_fills_what_nobody_writes(mok):
    """Under deterministic algorithms torch fills new memory: padding rows too hold the same from run to run."""
    torch.use_deterministic_algorithms(True)
    try:
        got = made(mok)["dispatch 0"]
    finally:
        torch.use_deterministic_algorithms(False)
    live = torch.zeros(got.rows, dtype=torch.bool, device="cuda")
    row, _, _ = ref.layout(routing("spread", 150, 3, 2)[0], 3)
    live[row.flatten().cuda()] = True
    assert (got.q[~live] == 0xFF).all() and torch.isnan(got.s[:, :got.rows][:, ~live]).all() and torch.isfinite(got.s[:, :got.rows][:, live]).all()
