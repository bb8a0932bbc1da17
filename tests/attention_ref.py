"""Plain 64-bit definitions of the attention operators, on the CPU, written
from the formulas of include/ar.h: norms with rotation and their gradient, the
4-bit cache's codes and places, and attention over it."""
from __future__ import annotations

import math

import numpy as np
import torch

LADDER = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def pairs(rotated: int, interleaved: bool):
    i = torch.arange(rotated // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotated // 2)


def norm_rope(x, w, cos_sin, eps, interleaved):
    """x (T, H, D), cos_sin (T, rotated) by token: (y, size): size bounds what
    the terms of y add up from."""
    x, w, cs = x.double(), w.double(), cos_sin.double()
    r = cs.shape[1]
    a, b = pairs(r, interleaved)
    z = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    y, size = z.clone(), z.abs()
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    y[..., a] = z[..., a] * c - z[..., b] * s
    y[..., b] = z[..., b] * c + z[..., a] * s
    both = z[..., a].abs() + z[..., b].abs()
    size[..., a] = both
    size[..., b] = both
    return y, size


def norm_rope_grad(gy, x, w, cos_sin, eps, interleaved):
    """(dx, its size, dw, its size)."""
    gy, x, w, cs = gy.double(), x.double(), w.double(), cos_sin.double()
    r = cs.shape[1]
    a, b = pairs(r, interleaved)
    g, gs = gy.clone(), gy.abs()
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    g[..., a] = gy[..., a] * c + gy[..., b] * s
    g[..., b] = gy[..., b] * c - gy[..., a] * s
    both = gy[..., a].abs() + gy[..., b].abs()
    gs[..., a] = both
    gs[..., b] = both
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * inv
    h, hs = g * w, gs * w.abs()
    dx = inv * (h - n * (h * n).mean(-1, keepdim=True))
    size = inv * (hs + n.abs() * (hs * n.abs()).mean(-1, keepdim=True))
    return dx, size, (g * n).sum((0, 1)), (gs * n.abs()).sum((0, 1))


# ------------------------------------------------------------------- the cache

def quantise(x):
    """x (..., D) as codes (..., D) and scale bytes (..., D / 32)."""
    y = x.double().numpy().reshape(*x.shape[:-1], -1, 32)
    most = np.abs(y).max(-1)
    byte = np.full(most.shape, 2, dtype=np.int64)
    with np.errstate(invalid="ignore"):
        for e in range(2, 252):
            byte[most >= 7 * 2.0 ** (e - 127)] = e + 1
        mag = np.abs(y) / 2.0 ** (byte[..., None] - 127)
        far = np.abs(mag[..., None] - LADDER)
        nearest = far.min(-1, keepdims=True)
        code = np.zeros(mag.shape, dtype=np.int64)
        for n in (1, 3, 5, 7, 0, 2, 4, 6):  # of two at one distance the even one stays
            code[far[..., n] == nearest[..., 0]] = n
    code += 8 * np.signbit(y)
    lost = ~np.isfinite(y).all(-1)
    byte[lost] = 255
    code[lost] = 0
    return code.reshape(x.shape), byte


def values(code, byte):
    v = LADDER[code & 7] * np.where(code >= 8, -1.0, 1.0)
    scale = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return v * np.repeat(scale, 32, axis=-1)


def places(D):
    """Byte of K code, V code (32, D) and K scale, V scale (32, D / 32) in a tile."""
    t, c, g = np.arange(32)[:, None], np.arange(D)[None], np.arange(D // 32)[None]
    W, G = D // 16, D // 32
    return (t * (D // 2) + c // 2,
            16 * D + ((t // 8 * 16 + c // W) * 8 + t % 8) * (W // 2) + c % W // 2,
            32 * D + (g * 16 + t // 8 * 4 + t % 4) * 2 + t % 8 // 4,
            33 * D + (t // 8 * G + g) * 8 + t % 8)


def pack(kc, kb, vc, vb):
    """Codes (pages, heads, tiles, 32, D) and scales (..., D / 32) as a cache."""
    D = kc.shape[-1]
    pk, pv, sk, sv = places(D)
    out = np.zeros((*kc.shape[:3], 34 * D), dtype=np.uint8)
    for p, code in ((pk, kc), (pv, vc)):
        out[..., p[:, 0::2]] = code[..., 0::2] | code[..., 1::2] << 4
    out[..., sk] = kb
    out[..., sv] = vb
    return out


def unpack(cache, D):
    """Codes and scales (pages, heads, tiles, 32, .) of a cache."""
    pk, pv, sk, sv = places(D)
    odd = np.arange(D) % 2 * 4
    return ((cache[..., pk] >> odd) & 15, cache[..., sk], (cache[..., pv] >> odd) & 15, cache[..., sv])


def attend(q, k, v, seen, scale):
    """q (M, D), k and v (N, D), seen (M, N): out, lse, and the sizes that
    errors are relative to: sum of weight |v|, and the largest over seen tokens
    of |q|_max |k|_1 scale."""
    q = q.double()
    k = torch.from_numpy(k)
    v = torch.from_numpy(v)
    M, N, D = q.shape[0], k.shape[0], q.shape[1]
    if N == 0:
        z = torch.zeros(M, D, dtype=torch.float64)
        return z, torch.full((M,), -math.inf, dtype=torch.float64), z, torch.zeros(M, dtype=torch.float64)
    s = torch.where(seen, (q @ k.T) * scale, torch.tensor(-math.inf, dtype=torch.float64))
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    # what a row does not see adds nothing, NaN or not
    used = seen.any(0)
    nan = torch.isnan(v) & used[:, None]
    clean = torch.nan_to_num(v, nan=0.0)
    out = p @ clean
    out[(seen.double() @ nan.double()) > 0] = math.nan
    reach = torch.where(used, torch.nan_to_num(k).abs().sum(1), 0.0).max() * q.abs().amax(1) * scale
    return out, lse, p @ clean.abs(), reach
