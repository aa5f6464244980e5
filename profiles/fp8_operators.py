"""Calls each of the routed-row and 8-bit operators once, for a capture of their kernels (profiles/fp8_operators.md)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_build_gb300 import mok  # noqa: E402


def n(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


# dense: 4096 x 7168 x 2048 forward, a row-scaled product of 2048 x 2048 over 8192 rows, 61 rows and one row
w, _ = mok.fp8_quantize_weight(n(7168, 2048))
a, _ = mok.fp8_quantize(n(4096, 2048))
mok.fp8_matmul(a, w)
_, xt = mok.fp8_quantize(n(8192, 2048), transposed=True)
mok.fp8_matmul(xt, xt, out_dtype=torch.float32)
mok.fp8_linear(n(61, 2048), w)
mok.fp8_linear(n(1, 2048), w)

# 16 experts of 2048 x 1024, 4096 tokens, top-4
T, E, K, H, N = 4096, 16, 4, 2048, 1024
ids = torch.rand((T, E), device="cuda").topk(K, 1).indices.to(torch.int32)
sched = mok.Routes(T, E, K).build(ids, torch.softmax(torch.randn((T, K), device="cuda"), 1))
we, wet = mok.fp8_quantize_weight(n(E, N, H), transposed=True)
x = n(T, H)
mok.dispatch_fp8(sched, x)
r, rt = mok.dispatch_fp8(sched, x, transposed=True)
y = mok.fp8_grouped_matmul(sched, r, we)
mok.combine(sched, y)
dr, _ = mok.combine_backward(sched, y, n(T, N))
d, dt = mok.fp8_quantize(dr, transposed=True, sched=sched)
mok.dispatch_backward(sched, mok.fp8_grouped_matmul(sched, d, wet))
mok.fp8_grouped_wgrad(sched, dt, rt)
mok.dispatch(sched, x)
torch.cuda.synchronize()
