"""Python's lock while a call waits for the GPU: a launch that finds the queue full must not hold up other threads (a
loader's, or the one that the GPU's work is waiting for)."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("call", ["norm", "norm_bwd", "dropout", "dropout_bwd", "ffn", "ffn_bwd"])
def test_other_threads_run_while_a_launch_waits(call):
    """3000 calls behind about a second of GPU work: more launches than the queue holds, so that some wait."""
    from mixture_experts_layer_build_gb300 import mok
    x, w, g, d = (torch.ones(s, dtype=BF, device="cuda") for s in ((1, 64), (64,), (32, 64), (64, 32)))
    rstd, drop = torch.ones(1, device="cuda"), mok.Dropout(0.1, torch.tensor([1, 2], device="cuda"))
    plan = mok.FFN(1, 64, 32)
    run = dict(norm=lambda: mok.rmsnorm_forward(x, w, 1e-6), norm_bwd=lambda: mok.rmsnorm_backward(x, rstd, w, x),
               dropout=lambda: mok.dropout_forward(x, drop), dropout_bwd=lambda: mok.dropout_backward(x, drop),
               ffn=lambda: plan.forward(x, g, g, d), ffn_bwd=lambda: plan.backward(x, g, g, d, x))[call]
    plan.forward(x, g, g, d)
    run()
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), []

    def tick():
        last = time.monotonic()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.monotonic()
            gaps.append(now - last)
            last = now
    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(2_000_000_000)  # cycles: about a second
        longest = 0.0
        for _ in range(3000):
            t0 = time.monotonic()
            run()
            longest = max(longest, time.monotonic() - t0)
    finally:
        stop.set()
        other.join()
    torch.cuda.synchronize()
    assert longest > 0.4, longest  # a call did wait
    assert max(gaps) < longest / 2, (max(gaps), longest)  # the lock was not held while it did
