"""Plain 64-bit definitions of the operators around a block, written from the
formulas of include/ar.h.  Each result comes with its size: what it adds up from,
in magnitudes, which errors of binary32 are relative to."""
from __future__ import annotations

import torch


def _mean(x):
    return x.mean(-1, keepdim=True)


def block_norm(parts, x, post, gate, pre, scale, eps):
    """parts: list of (T, D): ((h, size), (z, size)), or one pair without pre."""
    parts, x = [p.double() for p in parts], x.double()
    y = sum(parts[1:], parts[0])
    ys = sum(p.abs() for p in parts)
    u, us = y, ys
    if post is not None:
        r = 1 / torch.sqrt(_mean(y * y) + eps)
        u = y * r * post.double()
        # the root is off by what the sum is off by, in the mean
        spread = torch.sqrt(_mean(ys * ys) / (_mean(y * y) + eps))
        us = ys * r * post.double().abs() + u.abs() * spread
    g = torch.ones(()) if gate is None else gate.double()
    h = scale * x + g * u
    hs = (scale * x).abs() + g.abs() * us
    if pre is None:
        return [(h, hs)]
    r = 1 / torch.sqrt(_mean(h * h) + eps)
    z = h * r * pre.double()
    zs = hs * r * pre.double().abs() + z.abs() * torch.sqrt(_mean(hs * hs) / (_mean(h * h) + eps))
    return [(h, hs), (z, zs)]


def block_norm_grad(dh, dz, y, x, post, gate, pre, scale, eps):
    """dict of (gradient, size): dx, dy, and gate, post, pre where they are there
    (a gate (D) and both weights: sums over tokens)."""
    y, x = y.double(), x.double()
    r1 = 1 / torch.sqrt(_mean(y * y) + eps) if post is not None else torch.ones(())
    n1 = y * r1
    w1 = torch.ones(()) if post is None else post.double()
    g = torch.ones(()) if gate is None else gate.double()
    u = n1 * w1
    h, hs = scale * x + g * u, (scale * x).abs() + (g * u).abs()
    e = torch.zeros_like(x) if dh is None else dh.double()
    es = e.abs()
    out = {}
    if pre is not None:
        dz = dz.double()
        r2 = 1 / torch.sqrt(_mean(h * h) + eps)
        spread = torch.sqrt(_mean(hs * hs) / (_mean(h * h) + eps))
        n2, ns = h * r2, hs * r2 + (h * r2).abs() * spread
        q = dz * pre.double()
        e = e + r2 * (q - n2 * _mean(q * n2))
        es = es + r2 * (1 + spread) * (q.abs() + ns * _mean(q.abs() * ns))
        out["pre"] = ((dz * n2).sum(0), (dz.abs() * ns).sum(0))
    out["dx"] = (scale * e, abs(scale) * es)
    if gate is not None:
        dg, gs = e * u, es * u.abs()
        out["gate"] = (dg.sum(0), gs.sum(0)) if gate.dim() == 1 else (dg, gs)
    p, ps = e * g, es * g.abs()
    if post is None:
        out["dy"] = (p, ps)
        return out
    out["post"] = ((p * n1).sum(0), (ps * n1.abs()).sum(0))
    p, ps = p * w1, ps * w1.abs()
    out["dy"] = (r1 * (p - n1 * _mean(p * n1)), r1 * (ps + n1.abs() * _mean(ps * n1.abs())))
    return out
