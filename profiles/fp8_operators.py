"""Calls one of the routed-row or 8-bit operators once, for a capture of its kernel (profiles/fp8_operators.md).

Usage: python profiles/fp8_operators.py NAME; without a name the names, each with its kernel."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

KERNELS = {"linear_4096": "fp8_pair", "matmul_row_scaled": "fp8_pair", "linear_61": "fp8_tile", "linear_1": "fp8_tile",
           "quantize_weight": "fp8_quantize", "quantize_weights": "fp8_quantize", "quantize": "fp8_quantize",
           "quantize_both": "fp8_quantize", "quantize_routed": "fp8_quantize", "dispatch_fp8": "fp8_dispatch",
           "dispatch_fp8_both": "fp8_quantize", "experts": "fp8_pair", "experts_dx": "fp8_pair", "experts_dw": "fp8_pair",
           "dispatch": "gather_tokens", "dispatch_backward": "combine_kernel", "combine": "combine_kernel",
           "combine_backward": "combine_backward"}


def n(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def run(name: str):
    """The operator once, after what it needs; of its kernel it makes one launch."""
    from mixture_experts_layer_build_gb300 import mok
    blocks = lambda *s: mok.Fp8(torch.randint(0, 0x7F, s, device="cuda", dtype=torch.uint8),  # noqa: E731
                                torch.ones((*s[:-2], s[-2] // 128, s[-1] // 128), device="cuda"), s[-1], True)
    if name == "linear_4096":
        return mok.fp8_linear(n(4096, 2048), blocks(7168, 2048))
    if name == "matmul_row_scaled":
        _, xt = mok.fp8_quantize(n(8192, 2048), transposed=True)
        return mok.fp8_matmul(xt, xt, out_dtype=torch.float32)
    if name in ("linear_61", "linear_1"):
        return mok.fp8_linear(n(int(name[7:]), 2048), blocks(7168, 2048))
    if name == "quantize_weight":
        return mok.fp8_quantize_weight(n(7168, 2048))
    if name in ("quantize", "quantize_both"):
        return mok.fp8_quantize(n(4096 if name == "quantize" else 8192, 2048), transposed=name == "quantize_both")
    # 16 experts of 2048 x 1024, 4096 tokens, top-4
    T, E, K, H, N = 4096, 16, 4, 2048, 1024
    if name == "quantize_weights":
        return mok.fp8_quantize_weight(n(E, N, H), transposed=True)
    ids = torch.rand((T, E), device="cuda").topk(K, 1).indices.to(torch.int32)
    sched = mok.Routes(T, E, K).build(ids, torch.softmax(torch.randn((T, K), device="cuda"), 1))
    R = sched.c.rpad_max
    if name == "dispatch":
        return mok.dispatch(sched, n(T, H))
    if name == "dispatch_backward":
        return mok.dispatch_backward(sched, n(R, H))
    if name == "combine":
        return mok.combine(sched, n(R, N))
    if name == "combine_backward":
        return mok.combine_backward(sched, n(R, N), n(T, N))
    if name in ("dispatch_fp8", "dispatch_fp8_both"):
        return mok.dispatch_fp8(sched, n(T, H), transposed=name == "dispatch_fp8_both")
    if name == "quantize_routed":
        return mok.fp8_quantize(n(R, N), transposed=True, sched=sched)
    if name == "experts":
        return mok.fp8_grouped_matmul(sched, mok.dispatch_fp8(sched, n(T, H))[0], blocks(E, N, H))
    d, dt = mok.fp8_quantize(n(R, N), transposed=True, sched=sched)
    if name == "experts_dx":
        return mok.fp8_grouped_matmul(sched, d, blocks(E, H, N))
    if name == "experts_dw":
        return mok.fp8_grouped_wgrad(sched, dt, mok.dispatch_fp8(sched, n(T, H), transposed=True, rows=False)[1])
    raise SystemExit(f"no operator {name}")


if __name__ == "__main__":
    if len(sys.argv) != 2 or sys.argv[1] not in KERNELS:
        print("\n".join(f"{k}: {v}" for k, v in KERNELS.items()))
        raise SystemExit(0 if len(sys.argv) == 1 else 2)
    run(sys.argv[1])
    torch.cuda.synchronize()
