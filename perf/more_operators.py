"""Cases of the routed operators and of the 8-bit products, each in two forms.

  dispatch, dispatch_train  token rows sorted by expert into the schedule's padded layout, and the
                            gradient that sums a token's rows again
  combine, combine_train    a token's rows added up under its router weights, and the gradients of the
                            rows and of the weights
  linear, linear_train      y = x W^T on E4M3 codes with one fp32 scale per 1 x 128 values of x and per 128 x 128
                            values of W; with the gradients of x and W, whose operands are quantised along the
                            axis that is summed
  experts, experts_train    the same product for every expert's rows: tokens dispatched as E4M3 codes, one
                            matrix per expert; with both gradients, the tokens' summed over their rows

Scale of a block: max(amax, 2^-50) / 448 in fp32; codes: E4M3 of v * (448 / max(amax, 2^-50)).

`run` computes the plain form in elementary torch operations where `own` is false, and calls the
library where it is true; `exact` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False
ROW_TILE = 128      # each expert's rows are padded to a multiple of it
BLOCK = 128         # values that share a scale
LEAST = 2.0 ** -50  # of a block's largest magnitude


def listed():
    return [
        # one decoded token's rows on their way to its experts: latency only
        dict(name="dispatch_token", op="dispatch", T=1, E=128, K=8, H=4096, zipf=1.0),
        # a training step's rows there, and their gradients back: sizes that fill nothing evenly
        dict(name="dispatch_train_ragged", op="dispatch_train", T=1003, E=60, K=5, H=2056, zipf=0.5),
        # a prompt's expert outputs back to its tokens: a 64-expert layer
        dict(name="combine_4k", op="combine", T=4096, E=64, K=6, H=2048, zipf=0.0),
        # the same with the gradients of rows and router weights: the layer sweep's batch
        dict(name="combine_train_8k", op="combine_train", T=8192, E=128, K=8, H=4096, zipf=1.0),
        # one decoded token through a projection of the widest layer: weights' bytes and latency
        dict(name="linear_token", op="linear", M=1, N=2048, K=7168),
        # a batch of decoded tokens, one for each of 61 requests
        dict(name="linear_batch_61", op="linear", M=61, N=7168, K=2048),
        # a prompt
        dict(name="linear_prompt_4k", op="linear", M=4096, N=7168, K=2048),
        # training on sizes that fill no tile: forward, both gradients, all quantisation
        dict(name="linear_train_ragged", op="linear_train", M=1003, N=1000, K=2056),
        # training at the layer sweep's sizes
        dict(name="linear_train_8k", op="linear_train", M=8192, N=1536, K=4096),
        # one decoded token through one projection of its experts
        dict(name="experts_token", op="experts", T=1, E=128, K=8, H=4096, N=1536, zipf=1.0),
        # the layer sweep's batch through it, under its uneven routing
        dict(name="experts_8k", op="experts", T=8192, E=128, K=8, H=4096, N=1536, zipf=1.0),
        # a training step of it in a 64-expert layer
        dict(name="experts_train_4k", op="experts_train", T=4096, E=64, K=6, H=2048, N=1024, zipf=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_train", "combine", "combine_train", "linear", "linear", "linear_train",
                     "experts", "experts", "experts_train"])
    while True:
        if op in ("linear", "linear_train"):
            M = _log_int(rng, 1, 8192) if op == "linear" else _log_int(rng, 16, 8192)
            N, K = 8 * _log_int(rng, 8, 896), 8 * _log_int(rng, 8, 896)
            if N * K <= 7168 * 4096 and M * N * K <= 8192 * 4096 * 1536:
                return dict(op=op, M=M, N=N, K=K)
            continue
        T = _log_int(rng, 16 if op == "experts_train" else 1, 8192)
        E = _log_int(rng, 2, 256)
        K = rng.randint(1, min(E, 8))
        H, zipf = 8 * _log_int(rng, 16, 896), rng.choice([0.0, 0.5, 1.0, 2.0])
        if op in ("experts", "experts_train"):
            N = 8 * _log_int(rng, 16, 512)
            if E * N * H > 64 * 2048 * 1024 or T * K * N * H > 65536 * 4096 * 512:
                continue
            return dict(op=op, T=T, E=E, K=K, H=H, N=N, zipf=zipf)
        if T * K * H <= 65536 * 4096:
            return dict(op=op, T=T, E=E, K=K, H=H, zipf=zipf)


# -------------------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------------------
def _rows_max(case):
    """Rows of the layout that any routing of T * K slots over E experts fits in."""
    return case["T"] * case["K"] + case["E"] * (ROW_TILE - 1)


def _route(case, g):
    """Router's choice: K experts of E for each token, by Zipf popularity, and the softmax over their scores."""
    T, E, K = case["T"], case["E"], case["K"]
    popular = -case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp(1e-9, 1 - 1e-6)))
    score, ids = torch.topk(popular + noise, K, dim=1)
    e = torch.exp(score - score[:, :1])
    return ids.to(torch.int32), e / e.sum(1, keepdim=True)


def _layout(ids, E):
    """The schedule's tables: the row of each slot (a stable sort by expert, segments padded to 128 rows), the token of
    each row (-1 on padding), and on the host each expert's first row and rows."""
    T, K = ids.shape
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + ROW_TILE - 1) // ROW_TILE * ROW_TILE
    first, start = torch.cumsum(padded, 0) - padded, torch.cumsum(counts, 0) - counts
    order = torch.argsort(flat, stable=True)
    row = torch.empty_like(flat)
    row[order] = torch.arange(T * K, device=ids.device) - start[flat[order]] + first[flat[order]]
    token = torch.full((T * K + E * (ROW_TILE - 1),), -1, device=ids.device, dtype=torch.long)
    token[row] = torch.arange(T * K, device=ids.device) // K
    return dict(row=row.view(T, K), token=token, segments=list(zip(first.tolist(), counts.tolist())))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    op = case["op"]
    s = dict(case=case)
    if op in ("linear", "linear_train"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = n(M, K).to(bf)
        w = (n(N, K) * 0.02).to(bf)
        if op == "linear_train":
            s["w"], s["dy"] = w, n(M, N).to(bf)
        else:  # a checkpoint's codes and scales
            s["wq"], s["ws"] = _quantised(w.float(), (BLOCK, BLOCK))
            if own:
                s["w"] = _checkpoint(s["wq"], s["ws"])
        return s
    ids, wts = _route(case, g)
    rows = _rows_max(case)
    s["ids"], s["wts"], s["layout"] = ids, wts, _layout(ids, case["E"])
    token = s["layout"]["token"]
    H = case["H"]

    def layout_rows(width):  # what a kernel before this one left: zeros on padding rows
        r = n(rows, width).to(bf)
        return torch.where((token >= 0).unsqueeze(1), r, torch.zeros_like(r))

    if op in ("dispatch", "dispatch_train", "experts", "experts_train"):
        s["x"] = n(case["T"], H).to(bf)
    if op == "dispatch_train":
        s["drows"] = layout_rows(H)
    if op in ("combine", "combine_train"):
        s["rows"] = layout_rows(H)
    if op == "combine_train":
        s["dout"] = n(case["T"], H).to(bf)
    if op in ("experts", "experts_train"):
        w = (n(case["E"], case["N"], H) * 0.02).to(bf)
        if op == "experts_train":
            s["w"], s["dy"] = w, layout_rows(case["N"])
        else:
            s["wq"], s["ws"] = _quantised(w.float(), (BLOCK, BLOCK))
            if own:
                s["w"] = _checkpoint(s["wq"], s["ws"])
        del w
    if own:  # the step's schedule, and buffers that a program keeps: rows past the layout's last stay as they are
        from mixture_experts_layer_build_gb300 import mok
        s["routes"] = mok.Routes(case["T"], case["E"], case["K"])
        s["sched"] = s["routes"].build(ids, wts)
        if op in ("dispatch", "dispatch_train", "combine_train"):
            s["out"] = torch.zeros((rows, H), dtype=bf, device="cuda")
        elif op in ("experts", "experts_train"):
            s["out"] = torch.zeros((rows, case["N"]), dtype=bf, device="cuda")
    return s


def _checkpoint(q, scales):
    """Codes [.., N, K] and scales [.., N / 128, K / 128] as the library takes them: rows start on 16 bytes."""
    from mixture_experts_layer_build_gb300 import mok
    K = q.shape[-1]
    ld = (K + 15) // 16 * 16
    codes = torch.zeros((*q.shape[:-1], ld), dtype=torch.uint8, device=q.device)
    codes[..., :K] = q.view(torch.uint8)
    return mok.Fp8(codes, scales, K, block=True)


# -------------------------------------------------------------------------------------------------
# plain forms
# -------------------------------------------------------------------------------------------------
def _blocks(v, block):
    """[.., R, C] as [.., R / a, a, C / b, b], zeros past the edges."""
    (a, b), (R, C) = block, v.shape[-2:]
    ra, cb = -(-R // a), -(-C // b)
    if (ra * a, cb * b) != (R, C):
        p = v.new_zeros((*v.shape[:-2], ra * a, cb * b))
        p[..., :R, :C] = v
        v = p
    return v.reshape(*v.shape[:-2], ra, a, cb, b)


def _quantised(v, block):
    """E4M3 codes of fp32 values [.., R, C] and their scales [.., R / a, C / b]."""
    R, C = v.shape[-2:]
    t = _blocks(v, block)
    amax = t.abs().amax((-3, -1), keepdim=True).clamp(min=LEAST)
    most = torch.full_like(amax, 448.0)  # (a tensor: divided by, not multiplied with a reciprocal)
    q = (t * torch.div(most, amax)).clamp(-448, 448).to(torch.float8_e4m3fn)
    q = q.reshape(*v.shape[:-2], t.shape[-4] * block[0], t.shape[-2] * block[1])[..., :R, :C].contiguous()
    return q, torch.div(amax, most).squeeze(-1).squeeze(-2)


def _values(q, scales, block):
    """What codes and scales stand for, in fp32."""
    R, C = q.shape[-2:]
    t = _blocks(q.float(), block) * scales.unsqueeze(-2).unsqueeze(-1)
    return t.reshape(*q.shape[:-2], t.shape[-4] * block[0], t.shape[-2] * block[1])[..., :R, :C]


def _rounded(v, block=(1, BLOCK)):
    return _values(*_quantised(v.float(), block), block)


def _gathered(s):
    token = s["layout"]["token"]
    r = s["x"][token.clamp(min=0)]
    return torch.where((token >= 0).unsqueeze(1), r, torch.zeros_like(r))


def _summed(rows, row):
    """Per token the fp32 sum of its K rows."""
    acc = torch.zeros((row.shape[0], rows.shape[1]), dtype=torch.float32, device=rows.device)
    for k in range(row.shape[1]):
        acc = acc + rows[row[:, k]].float()
    return acc


def _plain(s):
    c = s["case"]
    op, bf = c["op"], torch.bfloat16
    if op == "linear":
        return dict(y=(_rounded(s["x"]) @ _values(s["wq"], s["ws"], (BLOCK, BLOCK)).T).to(bf))
    if op == "linear_train":
        w = _rounded(s["w"], (BLOCK, BLOCK))
        return dict(y=(_rounded(s["x"]) @ w.T).to(bf), dx=(_rounded(s["dy"]) @ w).to(bf),
                    dw=_rounded(s["dy"].T) @ _rounded(s["x"].T).T)
    L = s["layout"]
    if op == "dispatch":
        return dict(rows=_gathered(s))
    if op == "dispatch_train":
        return dict(rows=_gathered(s), dx=_summed(s["drows"], L["row"]).to(bf))
    if op in ("combine", "combine_train"):
        T, K = L["row"].shape
        acc = torch.zeros((T, c["H"]), dtype=torch.float32, device="cuda")
        for k in range(K):
            acc = acc + s["wts"][:, k:k + 1] * s["rows"][L["row"][:, k]].float()
        r = dict(out=acc.to(bf))
        if op == "combine_train":
            d = s["dout"].float()
            drows, dw = torch.zeros_like(s["rows"]), []
            for k in range(K):
                at = L["row"][:, k]
                drows[at] = (s["wts"][:, k:k + 1] * d).to(bf)
                dw.append((s["rows"][at].float() * d).sum(1))
            r.update(drows=drows, dw=torch.stack(dw, 1))
        return r
    x = _gathered(s)
    w = _rounded(s["w"], (BLOCK, BLOCK)) if op == "experts_train" else _values(s["wq"], s["ws"], (BLOCK, BLOCK))
    y = torch.zeros((x.shape[0], c["N"]), dtype=bf, device="cuda")
    xr = _rounded(x)
    for e, (r0, rn) in enumerate(L["segments"]):
        y[r0:r0 + rn] = (xr[r0:r0 + rn] @ w[e].T).to(bf)
    if op == "experts":
        return dict(y=y)
    del xr
    dr, dt, xt = _rounded(s["dy"]), _rounded(s["dy"].T), _rounded(x.T)
    dxr = torch.zeros_like(x)
    dw = torch.zeros((c["E"], c["N"], c["H"]), dtype=torch.float32, device="cuda")
    for e, (r0, rn) in enumerate(L["segments"]):
        dxr[r0:r0 + rn] = (dr[r0:r0 + rn] @ w[e]).to(bf)
        dw[e] = dt[:, r0:r0 + rn] @ xt[:, r0:r0 + rn].T
    return dict(y=y, dx=_summed(dxr, L["row"]).to(bf), dw=dw)


# -------------------------------------------------------------------------------------------------
# the library's calls
# -------------------------------------------------------------------------------------------------
def _own(s):
    from mixture_experts_layer_build_gb300 import mok
    op = s["case"]["op"]
    if op == "linear":
        return dict(y=mok.fp8_linear(s["x"], s["w"]))
    if op == "linear_train":
        w, wt = mok.fp8_quantize_weight(s["w"], transposed=True)
        x, xt = mok.fp8_quantize(s["x"], transposed=True)
        y = mok.fp8_matmul(x, w)
        d, dt = mok.fp8_quantize(s["dy"], transposed=True)
        return dict(y=y, dx=mok.fp8_matmul(d, wt), dw=mok.fp8_matmul(dt, xt, out_dtype=torch.float32))
    sched = s["sched"]
    if op == "dispatch":
        return dict(rows=mok.dispatch(sched, s["x"], out=s["out"]))
    if op == "dispatch_train":
        return dict(rows=mok.dispatch(sched, s["x"], out=s["out"]), dx=mok.dispatch_backward(sched, s["drows"]))
    if op == "combine":
        return dict(out=mok.combine(sched, s["rows"]))
    if op == "combine_train":
        out = mok.combine(sched, s["rows"])
        drows, dw = mok.combine_backward(sched, s["rows"], s["dout"], drows=s["out"])
        return dict(out=out, drows=drows, dw=dw)
    if op == "experts":
        x, _ = mok.dispatch_fp8(sched, s["x"])
        return dict(y=mok.fp8_grouped_matmul(sched, x, s["w"], out=s["out"]))
    w, wt = mok.fp8_quantize_weight(s["w"], transposed=True)
    x, xt = mok.dispatch_fp8(sched, s["x"], transposed=True)
    y = mok.fp8_grouped_matmul(sched, x, w, out=s["out"])
    d, dt = mok.fp8_quantize(s["dy"], transposed=True, sched=sched)
    dx = mok.dispatch_backward(sched, mok.fp8_grouped_matmul(sched, d, wt))
    return dict(y=y, dx=dx, dw=mok.fp8_grouped_wgrad(sched, dt, xt))


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------------------------
# what a pass cannot do without
# -------------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * M * K + N * K + 2 * M * N, flops=2 * M * N * K)
    if op == "linear_train":  # x, dy, w; y, dx, dw in fp32
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * (M * K + M * N + N * K) + 2 * (M * N + M * K) + 4 * N * K, flops=6 * M * N * K)
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    R = T * K
    if op == "dispatch":
        return dict(bytes=2 * T * H + 2 * R * H + 8 * R, flops=0)
    if op == "dispatch_train":
        return dict(bytes=4 * (T * H + R * H) + 8 * R, flops=R * H)
    if op == "combine":
        return dict(bytes=2 * (R * H + T * H) + 8 * R, flops=2 * R * H)
    if op == "combine_train":  # rows, dout; out, the rows' gradient, the weights' gradient
        return dict(bytes=2 * (2 * R * H + 2 * T * H) + 12 * R, flops=5 * R * H)
    N = case["N"]
    hit = E * (1 - (1 - 1 / E) ** R) if T > 1 else K  # experts with a row (uniform routing)
    if op == "experts":
        return dict(bytes=2 * T * H + hit * N * H + 2 * R * N, flops=2 * R * N * H)
    # x, dy rows, weights; y rows, dx, weight gradients in fp32
    return dict(bytes=2 * T * H + 2 * R * N + 2 * E * N * H + 2 * R * N + 2 * T * H + 4 * E * N * H, flops=6 * R * N * H)


# -------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# -------------------------------------------------------------------------------------------------
def _exact_e4m3(v):
    """Nearest E4M3 value, ties to even: 3 bits behind the leading one, steps of 2^-9 below 2^-6."""
    a = v.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def _exact_rounded(v, axis):
    """Values of v [R, C] (64 bits) after their rounding in blocks of 128 along `axis`, or (None) of 128 x 128."""
    out = torch.empty_like(v)
    rows = BLOCK if axis in (None, 0) else v.shape[0]
    cols = BLOCK if axis in (None, 1) else v.shape[1]
    over = None if axis is None else (axis,)
    for r in range(0, v.shape[0], rows):
        for c in range(0, v.shape[1], cols):
            b = v[r:r + rows, c:c + cols]
            top = b.abs().max() if over is None else b.abs().amax(over, keepdim=True)
            top = torch.clamp(top, min=LEAST).float()
            most = torch.full_like(top, 448.0)
            up, down = torch.div(most, top), torch.div(top, most)  # the format's scales are fp32 numbers
            code = _exact_e4m3((b.float() * up).double())
            out[r:r + rows, c:c + cols] = code * down.double()
    return out


def _exact_weight(s, e=None):
    if "wq" in s:
        q, sc = (s["wq"], s["ws"]) if e is None else (s["wq"][e], s["ws"][e])
        big = sc.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        return q.float().double() * big[:q.shape[0], :q.shape[1]]
    w = s["w"] if e is None else s["w"][e]
    return _exact_rounded(w.double(), None)


def exact(case, seed):
    global own
    was, own = own, False  # inputs alone, without the library's handles
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op in ("linear", "linear_train"):
        x, w = s["x"].double(), _exact_weight(s)
        r = dict(y=torch.einsum("mk,nk->mn", _exact_rounded(x, 1), w))
        if op == "linear_train":
            dy = s["dy"].double()
            r.update(dx=torch.einsum("mn,nk->mk", _exact_rounded(dy, 1), w),
                     dw=torch.einsum("mn,mk->nk", _exact_rounded(dy, 0), _exact_rounded(x, 0)))
        return r
    T, E, K, H = case["T"], case["E"], case["K"], case["H"]
    rows = _rows_max(case)
    flat = s["ids"].reshape(-1)
    first, slots = [0], []  # each expert's first row and slots, in order
    for e in range(E):
        slots.append(torch.nonzero(flat == e).flatten())
        first.append(first[-1] + (len(slots[-1]) + ROW_TILE - 1) // ROW_TILE * ROW_TILE)
    place = torch.empty(T * K, dtype=torch.long, device="cuda")
    for e in range(E):
        place[slots[e]] = first[e] + torch.arange(len(slots[e]), device="cuda")
    new = lambda width: torch.zeros((rows, width), dtype=torch.float64, device="cuda")  # noqa: E731
    back = lambda v: v[place].view(T, K, -1).sum(1)  # noqa: E731
    if op in ("combine", "combine_train"):
        y = s["rows"].double()
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        at = place.view(T, K)
        for k in range(K):
            out.addcmul_(s["wts"][:, k, None].double(), y[at[:, k]])
        r = dict(out=out)
        if op == "combine_train":
            d, drows = s["dout"].double(), new(H)
            dw = torch.empty((T, K), dtype=torch.float64, device="cuda")
            for k in range(K):
                drows[at[:, k]] = d * s["wts"][:, k, None].double()
                dw[:, k] = torch.einsum("th,th->t", d, y[at[:, k]])
            r.update(drows=drows, dw=dw)
        return r
    x = new(H)
    x[place] = s["x"].double().repeat_interleave(K, 0)
    if op == "dispatch":
        return dict(rows=x)
    if op == "dispatch_train":
        return dict(rows=x, dx=back(s["drows"].double()))
    N = case["N"]
    y = new(N)
    train = op == "experts_train"
    xr = _exact_rounded(x, 1)
    if train:
        dy, dxr = s["dy"].double(), new(H)
        dr, dt, xt = _exact_rounded(dy, 1), _exact_rounded(dy, 0), _exact_rounded(x, 0)
        dw = torch.zeros((E, N, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        r0, r1 = first[e], first[e] + len(slots[e])
        if r0 == r1:
            continue
        w = _exact_weight(s, e)
        y[r0:r1] = xr[r0:r1] @ w.T
        if train:
            dxr[r0:r1] = dr[r0:r1] @ w
            dw[e] = torch.einsum("rn,rh->nh", dt[r0:r1], xt[r0:r1])
    return dict(y=y, dx=back(dxr), dw=dw) if train else dict(y=y)
