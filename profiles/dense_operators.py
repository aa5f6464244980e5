"""Calls each of the dense operators once, for a capture of their kernels (profiles/dense_operators.md)."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_build_gb300 import mok  # noqa: E402


def n(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


drop = mok.Dropout(0.1, torch.tensor([1, 2], device="cuda"))
x, r, w = n(8192, 4096), n(8192, 4096), n(4096)
o = mok.rmsnorm_forward(x, w, 1e-6, residual=r, dropout=drop, bf16=False, mx=True)
mok.rmsnorm_backward(o.h, o.rstd, w, x, dres=r, dropout=drop)
mok.dropout_forward(x, drop, residual=r)
mok.dropout_backward(r, drop)

T, H, I = 4096, 4096, 1536
wg, wu, wd, dy = n(I, H), n(I, H), n(H, I), n(T, H)
f = mok.FFN(T, H, I)
f.forward(x[:T], wg, wu, wd)
f.backward(x[:T], wg, wu, wd, dy)

H, I = 7168, 2048
weights = [(n(I, H), n(I, H), n(H, I)) for _ in range(2)]
tokens = n(61, H)
mok.FFN(61, H, I, train=False).forward(tokens, *weights[0])
mok.FFN(1, H, I, train=False).forward(tokens[:1], *weights[1])
torch.cuda.synchronize()
