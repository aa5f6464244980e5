"""Forms of the sublayer that test_gpu_sublayer.py does not take, against the same composition in 64 bits with autograd:
GELU, bf16 gradients of the shared expert, one token, no gradient of the stream's later uses.  Its tolerance."""
import pytest
import torch

import dense_ref as ref
from helpers import TOL_BF16, rel_err
from test_gpu_sublayer import _params

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("T,act,dw,stream,p,with_dh", [(200, "gelu", BF, BF, 0.2, False), (130, "gelu", torch.float32, torch.float32, 0.0, True),
                                                       (1, "silu", BF, torch.float32, 0.1, True)])
def test_sublayer_forms(T, act, dw, stream, p, with_dh):
    from mixture_experts_layer_build_gb300 import mok
    from mixture_experts_layer_build_gb300.sublayer import Params, Sublayer
    H, I, E, K, Is, eps, seed, offset = 256, 128, 4, 2, 136, 1e-5, 3, 9
    w = _params(H, I, E, Is, 100 + T)
    g = torch.Generator().manual_seed(T)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    branch, residual, dout, dh = n(T, H).to(BF), n(T, H).to(stream), n(T, H).to(BF), n(T, H).to(stream)
    P = Params(**{k: v.cuda() for k, v in w.items()})
    sub = Sublayer(T, H, I, E, K, Is, act=act, eps=eps, shared_dw_dtype=dw)
    drop = mok.Dropout(p, torch.tensor([seed, offset], device="cuda")) if p else None
    out, h = sub.forward(branch.cuda(), residual.cuda(), P, drop)
    dbranch, dres, grads = sub.backward(dout.cuda(), dh.cuda() if with_dh else None, P, drop)
    assert sub.device_status() == 0 and grads.s_gate.dtype == dw

    leaf = {k: v.double().requires_grad_() for k, v in w.items()}
    b, r = branch.double().requires_grad_(), residual.double().requires_grad_()
    factors = ref.dropped(torch.ones(T, H, dtype=torch.float64), p, seed, offset) if p else 1.0
    hr = r + factors * b
    y, _ = ref.rmsnorm(hr, leaf["w_norm"], eps)
    ids = sub.ids.cpu().long()  # as the GPU chose them
    s = torch.softmax(torch.gather(y @ leaf["w_router"], 1, ids), 1)
    o = ref.ffn(y, leaf["s_gate"], leaf["s_up"], leaf["s_down"], act)[0]
    for k in range(K):
        a = torch.einsum("th,tih->ti", y, leaf["w_gate"][ids[:, k]])
        u = torch.einsum("th,tih->ti", y, leaf["w_up"][ids[:, k]])
        o = o + s[:, k:k + 1] * torch.einsum("ti,thi->th", ref.act(a, "silu")[0] * u, leaf["w_down"][ids[:, k]])
    loss = (o * dout.double()).sum()
    (loss + (hr * dh.double()).sum() if with_dh else loss).backward()
    for name, got, want in (("out", out, o), ("h", h, hr), ("dbranch", dbranch, b.grad), ("dresidual", dres, r.grad),
                            *((k, getattr(grads, k), t.grad) for k, t in leaf.items())):
        assert rel_err(got.detach().float().cpu().double().numpy(), want.detach().numpy()) <= TOL_BF16, name
