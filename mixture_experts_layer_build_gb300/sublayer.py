"""One transformer sublayer on the routed experts, forward and backward, from the library's calls:

    h   = residual + dropout(branch)          the residual stream, bf16 or fp32
    y   = rmsnorm(h) * w_norm
    out = routed_experts(y) + shared_expert(y)

`branch` is the previous sublayer's output, `out` this one's: the next sublayer's branch.  The
routed experts are the layer (router, schedule, expert GEMMs, combine), the shared expert the dense gated
feed-forward block, which adds the routed experts' output in its last epilogue; backward, it adds the
layer's and the router's share of dy in its own.  No arithmetic happens here.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import mok


@dataclass
class Params:
    w_norm: torch.Tensor              # [H] bf16
    w_router: torch.Tensor            # [H, E] bf16
    w_gate: torch.Tensor              # routed experts: [E, I, H], [E, I, H], [E, H, I] bf16
    w_up: torch.Tensor
    w_down: torch.Tensor
    s_gate: torch.Tensor              # shared expert: [Is, H], [Is, H], [H, Is] bf16
    s_up: torch.Tensor
    s_down: torch.Tensor


@dataclass
class ParamGrads:
    w_norm: torch.Tensor              # fp32
    w_router: torch.Tensor            # fp32
    w_gate: torch.Tensor              # fp32, as the layer gives them
    w_up: torch.Tensor
    w_down: torch.Tensor
    s_gate: torch.Tensor              # shared_dw_dtype
    s_up: torch.Tensor
    s_down: torch.Tensor


class Sublayer:
    """Buffers and plans for T tokens, E experts of [I, H] of which each token takes K, and a shared expert
    of [shared_I, H].  cfg: the layer's configuration (bf16 precision).  out and the experts' gradients are the plans' own
    buffers, overwritten by the next call."""

    def __init__(self, T: int, H: int, I: int, E: int, K: int, shared_I: int, act: str = "silu", eps: float = 1e-6,
                 cfg: mok.mok_config | None = None, shared_dw_dtype=torch.float32, device="cuda"):
        if cfg is not None and cfg.precision != mok.MOK_BF16:
            raise ValueError("cfg must be of MOK_BF16 precision: the parameters are bf16")
        self.K, self.eps = K, eps
        self.layer = mok.Layer(T, H, I, E, K, cfg or mok.make_config(0, 0), device)
        self.ffn = mok.FFN(T, H, shared_I, act=act, train=True, dw_dtype=shared_dw_dtype, device=device)

    def _here(self, x: torch.Tensor, name: str, p: Params):
        """Refuses tensors on another device than the plans': the layer's calls take their addresses as they are."""
        for k, t in ((name, x), *vars(p).items()):
            if t.device != self.ffn.out.device:
                raise ValueError(f"{k} must be on {self.ffn.out.device}, as the sublayer's buffers are, got {t.device}")

    def forward(self, branch: torch.Tensor, residual: torch.Tensor, p: Params, dropout: mok.Dropout | None = None,
                stream=None):
        """(out, h): this sublayer's output [T, H] bf16 and the residual stream, of residual's type."""
        self._here(branch, "branch", p)
        with mok._on_stream(stream, branch):
            self.norm = mok.rmsnorm_forward(branch, p.w_norm, self.eps, residual=residual, dropout=dropout)
            y = self.norm.y
            _, self.ids, self.weights = mok.router_forward(y, p.w_router, None, self.K)
            self.layer.schedule(self.ids, self.weights)
            routed = self.layer.forward(y, mok.weights_struct(p.w_gate, p.w_up, p.w_down))
            out = self.ffn.forward(y, p.s_gate, p.s_up, p.s_down, residual=routed)
        return out, self.norm.h

    def backward(self, dout: torch.Tensor, dh: torch.Tensor | None, p: Params, dropout: mok.Dropout | None = None,
                 stream=None):
        """(dbranch, dresidual, ParamGrads) of the last forward, for dout [T, H] bf16 = dL/dout and dh = dL/dh
        from the stream's later uses (None: 0).  dropout: the forward's, with its generator state unchanged."""
        self._here(dout, "dout", p)
        with mok._on_stream(stream, dout):
            y = self.norm.y
            g = self.layer.backward(dout, mok.weights_struct(p.w_gate, p.w_up, p.w_down))
            dw_router, _, dy = mok.router_backward(self.layer.sched, y, p.w_router, self.ids, self.weights,
                                                   g.d_topk_weights, dx=g.dx)
            f = self.ffn.backward(y, p.s_gate, p.s_up, p.s_down, dout, dx_add=dy)
            n = mok.rmsnorm_backward(self.norm.h, self.norm.rstd, p.w_norm, f.dx, dres=dh, dropout=dropout)
        return n.dx, n.dh, ParamGrads(n.dweight, dw_router, g.dw_gate, g.dw_up, g.dw_down, f.dw_gate, f.dw_up,
                                      f.dw_down)

    def device_status(self) -> int:
        """Bits (1 << status code) of the layer's and the shared expert's device status, after all work on their device,
        on whatever stream; synchronises."""
        return self.ffn.device_status() | mok.mok_read_device_status(self.layer.sched)
