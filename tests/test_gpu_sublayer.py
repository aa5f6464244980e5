"""The sublayer of sublayer.py -- dropout, residual, norm, router, routed experts, shared expert -- against the
same composition in 64 bits with autograd, at the routing that the GPU chose.

Tolerance: max |gpu - reference| / max |reference| per tensor within the layer's TOL_BF16 = 2e-2 (a chain
of bf16 tensors: y, a, dg and du are each rounded at 2^-8 and every output is a sum of many of them)."""
import pytest
import torch

import dense_ref as ref
from helpers import TOL_BF16, rel_err

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _params(H, I, E, Is, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: (torch.randn(s, generator=g) * 1.5 / H**0.5).to(BF)  # noqa: E731
    return dict(w_norm=(1 + 0.1 * torch.randn(H, generator=g)).to(BF), w_router=n(H, E), w_gate=n(E, I, H),
                w_up=n(E, I, H), w_down=n(E, H, I), s_gate=n(Is, H), s_up=n(Is, H), s_down=n(H, Is))


@pytest.mark.parametrize("T,stream,p", [(300, torch.float32, 0.1), (64, BF, 0.0)])
def test_sublayer_step(T, stream, p):
    from mixture_experts_layer_build_gb300 import mok
    from mixture_experts_layer_build_gb300.sublayer import Params, Sublayer
    H, I, E, K, Is, eps, seed, offset = 256, 128, 8, 2, 200, 1e-5, 11, 5
    w = _params(H, I, E, Is, T)
    g = torch.Generator().manual_seed(T + 1)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    branch, residual, dout, dh = n(T, H).to(BF), n(T, H).to(stream), n(T, H).to(BF), n(T, H).to(stream)
    P = Params(**{k: v.cuda() for k, v in w.items()})
    sub = Sublayer(T, H, I, E, K, Is, eps=eps)
    drop = mok.Dropout(p, torch.tensor([seed, offset], device="cuda")) if p else None
    out, h = sub.forward(branch.cuda(), residual.cuda(), P, drop)
    dbranch, dres, grads = sub.backward(dout.cuda(), dh.cuda(), P, drop)
    torch.cuda.synchronize()
    assert sub.device_status() == 0 and h.dtype == stream and dres.dtype == stream

    # the reference: every parameter and both inputs as leaves in fp64; routing ids as the GPU chose them
    leaf = {k: v.double().requires_grad_() for k, v in w.items()}
    b, r = branch.double().requires_grad_(), residual.double().requires_grad_()
    factors = ref.dropped(torch.ones(T, H, dtype=torch.float64), p, seed, offset) if p else 1.0
    hr = r + factors * b
    y, _ = ref.rmsnorm(hr, leaf["w_norm"], eps)
    ids = sub.ids.cpu().long()
    s = torch.softmax(torch.gather(y @ leaf["w_router"], 1, ids), 1)
    o = ref.ffn(y, leaf["s_gate"], leaf["s_up"], leaf["s_down"], "silu")[0]
    for k in range(K):
        a = torch.einsum("th,tih->ti", y, leaf["w_gate"][ids[:, k]])
        u = torch.einsum("th,tih->ti", y, leaf["w_up"][ids[:, k]])
        o = o + s[:, k:k + 1] * torch.einsum("ti,thi->th", ref.act(a, "silu")[0] * u, leaf["w_down"][ids[:, k]])
    ((o * dout.double()).sum() + (hr * dh.double()).sum()).backward()

    def near(got, want, name):
        assert rel_err(got.detach().float().cpu().double().numpy(), want.detach().numpy()) <= TOL_BF16, name
    near(out, o, "out")
    near(h, hr, "h")
    near(dbranch, b.grad, "dbranch")
    near(dres, r.grad, "dresidual")
    for k, t in leaf.items():
        near(getattr(grads, k), t.grad, k)
