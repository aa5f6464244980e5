"""Cases of the dense operators around the routed expert layer, each in two forms.

  norm, norm_bwd        root-mean-square norm of the residual stream after a branch is added to it,
                        with dropout on the branch, in bf16 and in MXFP8 (E4M3 codes, one E8M0 scale
                        per 32 values), and its gradient
  dropout, dropout_bwd  dropout from a counter-based generator, added to the residual stream, and
                        its gradient, from the same counters
  ffn, ffn_train        dense gated feed-forward block act(x Wg^T) * (x Wu^T) Wd^T (the shared expert
                        next to the routed ones), forward, and forward with every gradient

`run` computes the plain form in elementary torch operations where `own` is false, and calls the
library where it is true; `exact` is the definition in 64 bits.
"""
from __future__ import annotations

import functools
import math

import torch

own = False
EPS = 1e-6
ACTS = ("silu", "gelu")


def listed():
    return [
        # one decoded token: the norm before a layer, latency only
        dict(name="norm_token", op="norm", T=1, H=4096, f32=False, p=0.0, out="bf16"),
        # a training batch of the layer sweep's width into a block-scaled GEMM, dropout on the branch
        dict(name="norm_mx_8k", op="norm", T=8192, H=4096, f32=False, p=0.1, out="mx"),
        # a residual stream held in 32 bits; odd numbers of rows and of 8-value groups
        dict(name="norm_f32_ragged", op="norm", T=2051, H=2056, f32=True, p=0.0, out="bf16"),
        # its gradient in training: a 64-expert layer's width, dropout, the stream's own gradient
        dict(name="norm_bwd_4k", op="norm_bwd", T=4096, H=2048, f32=False, p=0.1),
        # the same with a 32-bit stream at the widest layer
        dict(name="norm_bwd_f32_16k", op="norm_bwd", T=16384, H=7168, f32=True, p=0.0),
        # dropout of a sublayer's output into the stream, without a norm behind it
        dict(name="dropout_8k", op="dropout", T=8192, H=4096, f32=False, p=0.1),
        # its gradient at the widest layer
        dict(name="dropout_bwd_16k", op="dropout_bwd", T=16384, H=7168, f32=False, p=0.2),
        # one decoded token through the shared expert
        dict(name="ffn_token", op="ffn", T=1, H=4096, I=1536, act="silu", residual=True),
        # a batch of decoded tokens, one for each of 61 requests, at the widest layer
        dict(name="ffn_batch_61", op="ffn", T=61, H=7168, I=2048, act="silu", residual=True),
        # a prompt
        dict(name="ffn_prompt_4k", op="ffn", T=4096, H=2048, I=1024, act="gelu", residual=False),
        # training at the layer sweep's sizes
        dict(name="ffn_train_8k", op="ffn_train", T=8192, H=4096, I=1536, act="silu", residual=True),
        # training on sizes that fill no tile
        dict(name="ffn_train_ragged", op="ffn_train", T=1003, H=2056, I=1000, act="gelu", residual=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "dropout", "dropout_bwd", "ffn", "ffn", "ffn_train"])
    if op in ("ffn", "ffn_train"):
        while True:
            T = _log_int(rng, 1, 16384) if op == "ffn" else _log_int(rng, 64, 8192)
            H, I = 8 * _log_int(rng, 32, 896), 8 * _log_int(rng, 16, 512)
            if T * H * I <= 8192 * 4096 * 1536 and H * I <= 7168 * 2048:
                return dict(op=op, T=T, H=H, I=I, act=rng.choice(ACTS), residual=rng.random() < 0.5)
    while True:
        T, f32, p = _log_int(rng, 1, 16384), rng.random() < 0.3, rng.choice([0.0, 0.05, 0.1, 0.5])
        out = rng.choice(["bf16", "mx", "both"])
        H = 32 * _log_int(rng, 4, 256) if op == "norm" and out != "bf16" else 8 * _log_int(rng, 16, 1024)
        if T * H > 16384 * 7168:
            continue
        c = dict(op=op, T=T, H=H, f32=f32, p=p)
        if op == "norm":
            c["out"] = out
        elif op != "norm_bwd":
            c["p"] = max(p, 0.05)
        return c


# -------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------
def _shape(case):
    return case["T"], case["H"], case.get("I", 0)


def prepare(case, seed):
    T, H, I = _shape(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    s = dict(case=case)
    if case["op"] in ("ffn", "ffn_train"):
        s["x"] = n(T, H).to(bf)
        s["wg"], s["wu"], s["wd"] = ((n(*d) * 0.02).to(bf) for d in ((I, H), (I, H), (H, I)))
        s["residual"] = n(T, H).to(bf) if case["residual"] else None
        if case["op"] == "ffn_train":
            s["dy"] = n(T, H).to(bf)
        if own:  # the block's plan: its context, workspace and outputs, kept between steps
            from mixture_experts_layer_build_gb300 import mok
            s["plan"] = mok.FFN(T, H, I, act=case["act"], train=case["op"] == "ffn_train")
        return s
    stream = torch.float32 if case["f32"] else bf
    s["rng"] = torch.randint(1 << 62, (2,), generator=g, device="cuda")  # the generator's seed and offset
    if case["op"] == "norm":
        s["x"], s["residual"] = n(T, H).to(bf), (n(T, H) * 2).to(stream)
        s["w"] = (1 + 0.1 * n(H)).to(bf)
    elif case["op"] == "norm_bwd":  # what the forward left: the stream h and 1 / rms of its rows
        s["h"] = (n(T, H) * 2).to(stream)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["w"] = (1 + 0.1 * n(H)).to(bf)
        s["dy"], s["dres"] = n(T, H).to(bf), n(T, H).to(stream)
    elif case["op"] == "dropout":
        s["x"], s["residual"] = n(T, H).to(bf), (n(T, H) * 2).to(stream)
    else:
        s["dout"] = n(T, H).to(stream)
    return s


# -------------------------------------------------------------------------------------------------
# plain forms
# -------------------------------------------------------------------------------------------------
M32 = 0xFFFFFFFF


def _round(mult, c, key):
    """One round of Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011)
    on the counters' even and odd words, [2, n] each: 32-bit words held in int64."""
    even, odd = c
    p = even * mult
    return ((p >> 32) & M32).flip(0) ^ odd ^ key.unsqueeze(1), (p & M32).flip(0)


def _threshold(p):
    return int(p * 65536 + 0.5)  # of a 16-bit draw: dropped below it


def _keep(rng, p, T, H):
    """Truth values [T, H]: Philox4x32-10 of counter (index of the 8-value group, offset) under key
    seed gives eight 16-bit draws, low halves first; a value is kept when its draw is >= 65536 p."""
    b = torch.arange(T * H // 8, device=rng.device)
    words = torch.stack([rng & M32, (rng >> 32) & M32])  # low and high words of seed and offset
    even = torch.stack([b & M32, words[0, 1].expand_as(b)])
    odd = torch.stack([(b >> 32) & M32, words[1, 1].expand_as(b)])
    n = torch.arange(2, device=rng.device)  # multipliers and key steps without a copy from the host
    mult = (0xD2511F53 + n * (0xCD9E8D57 - 0xD2511F53)).unsqueeze(1)
    weyl = 0x9E3779B9 + n * (0xBB67AE85 - 0x9E3779B9)
    keys = (words[:, 0] + torch.arange(10, device=rng.device).unsqueeze(1) * weyl) & M32
    even, odd = functools.reduce(functools.partial(_round, mult), keys, (even, odd))
    draws = torch.stack([even[0], odd[0], even[1], odd[1]], 1).unsqueeze(2)
    draws = torch.cat([draws & 0xFFFF, draws >> 16], 2)
    return (draws >= _threshold(p)).reshape(T, H)


def _dropped(v, rng, p):
    if p == 0:
        return v
    t = _threshold(p)
    return torch.where(_keep(rng, p, *v.shape), v * (65536 / (65536 - t)), torch.zeros_like(v))


def _mx(v):
    """MXFP8 of fp32 rows: codes (float8_e4m3fn) and scales (float8_e8m0fnu), one per 32 values."""
    T, H = v.shape
    b = v.reshape(T, H // 32, 32)
    _, e = torch.frexp(b.abs().amax(2))
    shared = torch.where(b.abs().amax(2) > 0, e - 9, torch.full_like(e, -127)).clamp(min=-127)
    q = (b * torch.exp2(-shared.float()).unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.reshape(T, H), (shared + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _act(g, act):
    """The activation and its derivative at g."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c, k = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (g + k * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * k * g * g)


def _plain(s):
    c = s["case"]
    op, p = c["op"], c.get("p", 0.0)
    bf = torch.bfloat16
    if op == "norm":
        h = (s["residual"].float() + _dropped(s["x"].float(), s["rng"], p)).to(s["residual"].dtype)
        hf = h.float()  # the norm is of the stream's stored values
        rstd = torch.rsqrt(hf.square().mean(1) + EPS)
        y = hf * rstd.unsqueeze(1) * s["w"].float()
        r = dict(h=h, rstd=rstd)
        if c["out"] != "mx":
            r["y"] = y.to(bf)
        if c["out"] != "bf16":
            r["q"], r["s"] = _mx(y)
        return r
    if op == "norm_bwd":
        xh = s["h"].float() * s["rstd"].unsqueeze(1)
        dy = s["dy"].float()
        g = dy * s["w"].float()
        dh = s["rstd"].unsqueeze(1) * (g - xh * (g * xh).mean(1, keepdim=True)) + s["dres"].float()
        r = dict(dh=dh.to(s["h"].dtype), dw=(dy * xh).sum(0))
        if p or c["f32"]:  # else the branch's gradient is the stream's
            r["dx"] = _dropped(dh, s["rng"], p).to(bf)
        return r
    if op == "dropout":
        return dict(out=(s["residual"].float() + _dropped(s["x"].float(), s["rng"], p)).to(s["residual"].dtype))
    if op == "dropout_bwd":
        return dict(dx=_dropped(s["dout"].float(), s["rng"], p).to(bf))
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.T, x @ wu.T
    f, df = _act(g, c["act"])
    a = f * u
    out = a @ wd.T
    if s["residual"] is not None:
        out = out + s["residual"].float()
    r = dict(out=out.to(bf))
    if op == "ffn_train":
        dy = s["dy"].float()
        da = dy @ wd
        dg, du = da * u * df, da * f
        r.update(dx=(dg @ wg + du @ wu).to(bf), dw_gate=(dg.T @ x).to(bf), dw_up=(du.T @ x).to(bf),
                 dw_down=(dy.T @ a).to(bf))
    return r


# -------------------------------------------------------------------------------------------------
# the library's calls
# -------------------------------------------------------------------------------------------------
def _own(s):
    from mixture_experts_layer_build_gb300 import mok
    c = s["case"]
    op, p = c["op"], c.get("p", 0.0)
    if op == "ffn":
        return dict(out=s["plan"].forward(s["x"], s["wg"], s["wu"], s["wd"], residual=s["residual"]))
    if op == "ffn_train":
        plan = s["plan"]
        out = plan.forward(s["x"], s["wg"], s["wu"], s["wd"], residual=s["residual"])
        g = plan.backward(s["x"], s["wg"], s["wu"], s["wd"], s["dy"])
        return dict(out=out, dx=g.dx, dw_gate=g.dw_gate, dw_up=g.dw_up, dw_down=g.dw_down)
    drop = mok.Dropout(p, s["rng"]) if p else None
    if op == "norm":
        o = mok.rmsnorm_forward(s["x"], s["w"], EPS, residual=s["residual"], dropout=drop, bf16=c["out"] != "mx",
                                mx=c["out"] != "bf16")
        r = dict(h=o.h, rstd=o.rstd)
        if o.y is not None:
            r["y"] = o.y
        if o.q is not None:
            r["q"], r["s"] = o.q.view(torch.float8_e4m3fn), o.s.view(torch.float8_e8m0fnu)
        return r
    if op == "norm_bwd":
        g = mok.rmsnorm_backward(s["h"], s["rstd"], s["w"], s["dy"], dres=s["dres"], dropout=drop)
        r = dict(dh=g.dh, dw=g.dweight)
        if p or c["f32"]:
            r["dx"] = g.dx
        return r
    if op == "dropout":
        return dict(out=mok.dropout_forward(s["x"], drop, residual=s["residual"]))
    return dict(dx=mok.dropout_backward(s["dout"], drop))


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------------
# what a pass cannot do without
# -------------------------------------------------------------------------------------------------
def work(case):
    T, H, I = _shape(case)
    op, n = case["op"], T * H
    if op in ("ffn", "ffn_train"):
        train = op == "ffn_train"
        w = 3 * H * I * 2
        tensors = 2 + (1 if case["residual"] else 0) + (2 if train else 0)  # x, out; residual; dy, dx
        return dict(bytes=n * 2 * tensors + w * (2 if train else 1), flops=(18 if train else 6) * n * I)
    st = 4 if case["f32"] else 2
    if op == "norm":
        y = {"bf16": 2.0, "mx": 33 / 32, "both": 2 + 33 / 32}[case["out"]]
        return dict(bytes=n * (2 + 2 * st + y) + 2 * H + 4 * T, flops=6 * n)
    if op == "norm_bwd":
        dx = 2 if case["p"] or case["f32"] else 0
        return dict(bytes=n * (2 + 3 * st + dx) + 6 * H + 4 * T, flops=12 * n)
    return dict(bytes=n * (2 + (2 if op == "dropout" else 1) * st), flops=2 * n)


# -------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------
def _exact_mask(state, p, T, H):
    """Factors [T, H]: 0, or 1 / (share kept); Philox4x32-10 over 32-bit words held in int64."""
    n = T * H // 8
    i = torch.arange(n, device=state.device)
    words = [i % 2**32, i // 2**32, (state[1] % 2**32).expand(n), (state[1] // 2**32).expand(n)]
    key = [state[0] % 2**32, state[0] // 2**32]

    def product(w, m):  # by 16-bit halves: nothing passes 2^63
        lo, hi = (w % 65536) * m, (w // 65536) * m
        mid = hi + lo // 65536
        return mid // 65536, (mid % 65536) * 65536 + lo % 65536

    for _ in range(10):
        ah, al = product(words[0], 0xD2511F53)
        bh, bl = product(words[2], 0xCD9E8D57)
        words = [bh ^ words[1] ^ key[0], bl, ah ^ words[3] ^ key[1], al]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    share = round(p * 65536)
    factor = torch.zeros(n, 8, dtype=torch.float64, device=state.device)
    for j in range(8):
        half = words[j // 2] // 65536 if j % 2 else words[j // 2] % 65536
        factor[:, j] = (half >= share).double() * (65536 / (65536 - share))
    return factor.view(T, H)


def exact(case, seed):
    s = prepare(case, seed)
    T, H, I = _shape(case)
    op, p = case["op"], case.get("p", 0.0)
    f = _exact_mask(s["rng"], p, T, H) if p else 1.0
    if op == "norm":
        h = s["residual"].double() + f * s["x"].double()
        stored = h.to(s["residual"].dtype).double()
        rms = torch.sqrt((stored * stored).sum(1) / H + EPS)
        y = s["w"].double() * stored / rms[:, None]
        r = dict(h=h, rstd=1 / rms)
        if case["out"] != "mx":
            r["y"] = y
        if case["out"] != "bf16":  # the scales, and the scaled values before they are rounded to codes
            top = y.view(T, H // 32, 32).abs().amax(2)
            scale = torch.exp2(torch.floor(torch.log2(top)) - 8)
            r["q"] = (y.view(T, H // 32, 32) / scale[:, :, None]).view(T, H)
            r["s"] = scale
        return r
    if op == "norm_bwd":
        h, rstd, w, dy = (s[k].double() for k in ("h", "rstd", "w", "dy"))
        along = ((dy * w) * h).sum(1) / H
        dh = s["dres"].double() + rstd[:, None] * dy * w - (rstd**3 * along)[:, None] * h
        r = dict(dh=dh, dw=torch.einsum("th,th,t->h", dy, h, rstd))
        if p or case["f32"]:
            r["dx"] = f * dh
        return r
    if op == "dropout":
        return dict(out=s["residual"].double() + f * s["x"].double())
    if op == "dropout_bwd":
        return dict(dx=f * s["dout"].double())
    x, wg, wu, wd = (s[k].double() for k in ("x", "wg", "wu", "wd"))
    g, u = torch.einsum("th,ih->ti", x, wg), torch.einsum("th,ih->ti", x, wu)
    if case["act"] == "silu":
        sig = torch.sigmoid(g)
        v, dv = g * sig, sig + g * sig * (1 - sig)
    else:  # 0.5 (1 + tanh z) = sigmoid(2 z)
        z2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g**3)
        sig = torch.sigmoid(z2)
        v = g * sig
        dv = sig + g * sig * (1 - sig) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g**2)
    a = v * u
    out = torch.einsum("ti,hi->th", a, wd)
    r = dict(out=out + s["residual"].double() if s["residual"] is not None else out)
    if op == "ffn_train":
        dy = s["dy"].double()
        da = torch.einsum("th,hi->ti", dy, wd)
        dg, du = da * u * dv, da * v
        r.update(dx=torch.einsum("ti,ih->th", dg, wg) + torch.einsum("ti,ih->th", du, wu),
                 dw_gate=torch.einsum("ti,th->ih", dg, x), dw_up=torch.einsum("ti,th->ih", du, x),
                 dw_down=torch.einsum("th,ti->hi", dy, a))
    return r
