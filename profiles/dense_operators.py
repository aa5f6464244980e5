"""Calls one of the dense operators once, for a capture of its kernels (profiles/dense_operators.md).

Usage: python profiles/dense_operators.py NAME; without a name the names, each with its kernels."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

KERNELS = {"rmsnorm_forward": "rmsnorm_fwd", "rmsnorm_backward": "rmsnorm_bwd or rmsnorm_dw", "dropout_forward": "dropout_kernel",
           "dropout_backward": "dropout_kernel", "ffn_train": "ffn_pair: gate/up, down, DACT, DX (-s 0 to 3)",
           "ffn_61": "ffn_tile: gate/up, down (-s 0, 1)", "ffn_1": "ffn_row: gate/up, down (-s 0, 1)"}


def n(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def run(name: str):
    from mixture_experts_layer_build_gb300 import mok
    if name == "ffn_train":
        T, H, I = 4096, 4096, 1536
        x, wg, wu, wd, dy = n(T, H), n(I, H), n(I, H), n(H, I), n(T, H)
        f = mok.FFN(T, H, I)
        f.forward(x, wg, wu, wd)
        return f.backward(x, wg, wu, wd, dy)
    if name in ("ffn_61", "ffn_1"):
        T, H, I = int(name[4:]), 7168, 2048
        return mok.FFN(T, H, I, train=False).forward(n(T, H), n(I, H), n(I, H), n(H, I))
    drop = mok.Dropout(0.1, torch.tensor([1, 2], device="cuda"))
    x, r, w = n(8192, 4096), n(8192, 4096), n(4096)
    if name == "rmsnorm_forward":
        return mok.rmsnorm_forward(x, w, 1e-6, residual=r, dropout=drop, bf16=False, mx=True)
    if name == "rmsnorm_backward":
        return mok.rmsnorm_backward(r, torch.ones(8192, device="cuda"), w, x, dres=r, dropout=drop)
    if name == "dropout_forward":
        return mok.dropout_forward(x, drop, residual=r)
    if name == "dropout_backward":
        return mok.dropout_backward(r, drop)
    raise SystemExit(f"no operator {name}")


if __name__ == "__main__":
    if len(sys.argv) != 2 or sys.argv[1] not in KERNELS:
        print("\n".join(f"{k}: {v}" for k, v in KERNELS.items()))
        raise SystemExit(0 if len(sys.argv) == 1 else 2)
    run(sys.argv[1])
    torch.cuda.synchronize()
