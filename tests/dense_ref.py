"""Plain 64-bit forms of the dense operators (dropout, norm, gated feed-forward block) for the tests,
on CPU tensors, written from the formulas in include/mok.h."""
import math

import numpy as np
import torch

RNG_M = (0xD2511F53, 0xCD9E8D57)
RNG_W = (0x9E3779B9, 0xBB67AE85)


def philox4x32_10(counter, key):
    """One block of Philox4x32-10 with Python integers: 4 counter words, 2 key words -> 4 words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = RNG_M[0] * c[0], RNG_M[1] * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + RNG_W[0]) & 0xFFFFFFFF, (k[1] + RNG_W[1]) & 0xFFFFFFFF]
    return c


def draws16(n, seed, offset, first_group=0):
    """The 16-bit draws of n values (a multiple of 8) from group first_group on, vectorised."""
    g = np.arange(n // 8, dtype=np.uint64) + np.uint64(first_group)
    lo = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    c = [g & lo, g >> s32, np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * np.uint64(RNG_M[0]), c[2] * np.uint64(RNG_M[1])
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + RNG_W[0]) & 0xFFFFFFFF, (k[1] + RNG_W[1]) & 0xFFFFFFFF]
    return np.stack([v for w in c for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(-1).astype(np.int64)


def threshold(p):
    return int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))


def keep(shape, p, seed, offset):
    n = int(np.prod(shape))
    return torch.from_numpy(draws16(n, seed, offset) >= threshold(p)).reshape(shape)


def dropped(v, p, seed, offset):
    """Factors applied to v (fp64): a dropped value is 0 whatever it holds."""
    t = threshold(p)
    if t >= 65536:
        return torch.zeros_like(v)
    return torch.where(keep(v.shape, p, seed, offset), v * (65536.0 / (65536 - t)), torch.zeros_like(v))


def rmsnorm(h, w, eps):
    rstd = 1.0 / torch.sqrt(h.square().mean(1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_grads(h, rstd, w, dy, dres):
    xh = h * rstd[:, None]
    g = dy * w
    dh = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    return (dh if dres is None else dh + dres), (dy * xh).sum(0)


def act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g**3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def ffn(x, wg, wu, wd, kind, residual=None):
    g, u = x @ wg.T, x @ wu.T
    f, df = act(g, kind)
    a = f * u
    out = a @ wd.T
    return (out if residual is None else out + residual), (g, u, f, df, a)


def ffn_grads(x, wg, wu, wd, dy, saved):
    g, u, f, df, a = saved
    da = dy @ wd
    dg, du = da * u * df, da * f
    return dict(dx=dg @ wg + du @ wu, dw_gate=dg.T @ x, dw_up=du.T @ x, dw_down=dy.T @ a), (dg, du)
