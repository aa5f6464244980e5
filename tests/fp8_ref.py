"""Plain 64-bit forms of the routed-row operators and of the 8-bit products (test infrastructure).

Quantisation is defined by fp32 steps (t = max(amax, 2^-50), up = 448 / t, scale = t / 448, v * up), each of them rounded
from its exact 64-bit value here: quotients and products of two fp32 numbers are rounded correctly through 64 bits."""
import torch

F64 = torch.float64
LEAST = 2.0**-50


def f32(v):
    return v.to(torch.float32).to(F64)


def e4m3(v):
    """Nearest E4M3 value (ties to even, saturating at 448) of each v, |v| finite."""
    a = v.abs()
    _, e = torch.frexp(a.clamp(min=2.0**-6))  # a in [2^(e-1), 2^e): 3 bits behind the leading one
    step = (e.to(torch.int64) + (1023 - 4) << 52).view(F64)  # 2^(e - 4) from its bits
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), v)


def decode(q):
    """E4M3 bytes (or float8 tensor) -> values."""
    return q.view(torch.float8_e4m3fn).to(torch.float32).to(F64)


def quantize(x, block):
    """(codes' values [R, C], scales [ceil(R/a), ceil(C/b)]) of x [R, C] in blocks of block = (a, b)."""
    x = x.to(F64)
    (R, C), (a, b) = x.shape, block
    nr, nc = -(-R // a), -(-C // b)
    p = torch.zeros((nr * a, nc * b), dtype=F64, device=x.device)
    p[:R, :C] = x
    p = p.view(nr, a, nc, b)
    bad = ~torch.isfinite(p).all(3, keepdim=True).all(1, keepdim=True)
    t = torch.where(torch.isfinite(p), p, torch.zeros_like(p)).abs().amax((1, 3), keepdim=True).clamp(min=LEAST)
    up, scale = f32(448.0 / t), f32(t / 448.0)
    nan = torch.full_like(t, float("nan"))
    q = torch.where(bad, nan, e4m3(f32(torch.where(bad, torch.zeros_like(p), p) * up)))
    return q.reshape(nr * a, nc * b)[:R, :C], torch.where(bad, nan, scale)[:, 0, :, 0]


def values(q, scales, block):
    """What codes (values [R, C]) under scales [ceil(R/a), ceil(C/b)] stand for."""
    R, C = q.shape
    big = scales.to(F64).repeat_interleave(block[0], 0).repeat_interleave(block[1], 1)
    return q.to(F64) * big[:R, :C]


def of(m, e=None):
    """What an Fp8 (matrix e of a batch) stands for, in 64 bits."""
    q, s = (m.q, m.s) if e is None else (m.q[e], m.s[e])
    q = decode(q)[:, :m.cols]
    return values(q, s, (128, 128)) if m.block else values(q, s[:, :q.shape[0]].T, (1, 128))


def layout(ids, E):
    """The schedule's layout, slot by slot: (row of each slot [T, K], -1 for an invalid id; each expert's (first row, rows);
    the layout's end)."""
    T, K = ids.shape
    ids = ids.cpu().tolist()
    mine = [[] for _ in range(E)]
    for t in range(T):
        for k in range(K):
            if 0 <= ids[t][k] < E:
                mine[ids[t][k]].append((t, k))
    row = torch.full((T, K), -1, dtype=torch.long)
    segments, at = [], 0
    for slots in mine:
        segments.append((at, len(slots)))
        for i, (t, k) in enumerate(slots):
            row[t, k] = at + i
        at += (len(slots) + 127) // 128 * 128
    return row, segments, at


def dispatch(x, row, rows):
    """[rows, W]: token t's row of x at each of its slots' rows, zeros elsewhere."""
    out = torch.zeros((rows, x.shape[1]), dtype=x.dtype, device=x.device)
    t, k = torch.nonzero(row >= 0, as_tuple=True)
    out[row[t, k].to(x.device)] = x[t.to(x.device)]
    return out


def combine(rows, row, w=None):
    """([T, W] sum of each token's rows times w, the sum of the magnitudes)."""
    T, K = row.shape
    out = torch.zeros((T, rows.shape[1]), dtype=F64, device=rows.device)
    mag = torch.zeros_like(out)
    for k in range(K):
        there = (row[:, k] >= 0).to(rows.device)
        v = rows[row[:, k].clamp(min=0).to(rows.device)].to(F64)
        if w is not None:
            v = v * w[:, k, None].to(F64)
        v = torch.where(there[:, None], v, torch.zeros_like(v))
        out, mag = out + v, mag + v.abs()
    return out, mag


def combine_grads(rows, dout, row, w):
    """(drows [rows, W], dw [T, K], the magnitudes behind dw)."""
    T, K = row.shape
    d = dout.to(F64)
    drows = torch.zeros(rows.shape, dtype=F64, device=rows.device)
    dw = torch.zeros((T, K), dtype=F64, device=rows.device)
    mag = torch.zeros_like(dw)
    for k in range(K):
        t = torch.nonzero(row[:, k] >= 0)[:, 0].to(rows.device)
        at = row[:, k].to(rows.device)[t]
        drows[at] = w[t, k, None].to(F64) * d[t]
        p = d[t] * rows[at].to(F64)
        dw[t, k], mag[t, k] = p.sum(1), p.abs().sum(1)
    return drows, dw, mag
