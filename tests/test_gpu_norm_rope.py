"""GPU parity of the head norms with rotation, and of their gradient, against
the 64-bit definitions.

Tolerances.  One rounding of the result to bf16, half a step: 2^-8 of it.  In
binary32 before it: a sum of up to 256 squares (2^-19 of it at most), its
reciprocal root, and fewer than ten operations: below 2^-18 of the terms that
the result adds up from, whose size the definitions return.  The weights'
gradients are binary32 sums of terms with that error; a lane adds at most some
hundred terms one after another, and the rest is a tree: 2^-16 of the sum of the
terms' sizes."""
from __future__ import annotations

import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8

CASES = [  # tokens, heads, kv_heads, dim, rotated, interleaved
    (1, 1, 1, 128, 128, False), (8, 8, 1, 128, 128, False), (3, 5, 2, 64, 64, False),
    (7, 40, 8, 64, 32, True), (5, 3, 0, 128, 48, False), (5, 0, 3, 128, 48, True),
    (2, 9, 4, 256, 256, False), (9, 2, 1, 256, 128, True), (4, 7, 7, 64, 16, False),
    (6, 1, 5, 128, 80, True), (1031, 12, 3, 128, 128, False), (17, 100, 11, 64, 64, True)]


def _inputs(T, hq, hk, D, r, seed, table=97, odd=False):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn(D, generator=g))
    pad = 1 if odd else 0  # an odd stride: no row after the first starts on 16 bytes
    qkv = torch.zeros(T, (hq + 2 * hk) * D + pad, dtype=torch.bfloat16)
    qkv[:, :(hq + 2 * hk) * D] = (torch.randn(T, hq + 2 * hk, D, generator=g) * size).reshape(T, -1).bfloat16()
    if T > 2:
        qkv[1] = 0  # a row of zeros
    w = [(1 + 0.3 * torch.randn(D, generator=g)).bfloat16() for _ in range(2)]
    angle = torch.rand(table, r // 2, generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    pos = torch.randint(0, table, (T,), generator=g)
    return qkv, w, cs, pos


def _views(qkv, hq, hk, D):
    x = qkv[:, :(hq + 2 * hk) * D].unflatten(1, (hq + 2 * hk, D))
    return x[:, :hq], x[:, hq:hq + hk]


def _close(got, want, size, rel, what):
    off = (got.cpu().double() - want).abs()
    tol = BF * want.abs() + rel * size + 1e-30
    assert bool((off <= tol).all()), f"{what}: {float((off / tol).max())} times the tolerance"


@pytest.mark.parametrize("T,hq,hk,D,r,inter", CASES)
@pytest.mark.parametrize("odd", [False, True])
def test_forward(T, hq, hk, D, r, inter, odd):
    announce(f"norm_rope {T} {hq} {hk} {D} {r} {inter} odd={odd}")
    qkv, w, cs, pos = _inputs(T, hq, hk, D, r, T + D, odd=odd)
    d = qkv.to(DEV)
    q, k = _views(d, hq, hk, D)
    qo = torch.full((T, hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, hk, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ar.ar_qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), cs.to(DEV), pos.to(DEV), qo, ko, eps=1e-5, interleaved=inter)
    for x, wt, o, n in zip(_views(qkv, hq, hk, D), w, (qo, ko), "qk"):
        if o.numel():
            want, size = R.norm_rope(x, wt, cs[pos], 1e-5, inter)
            _close(o, want, size, 2.0 ** -18, n)
    # in place, the values beside the keys untouched, the same bits
    ar.ar_qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), cs.to(DEV), pos.to(DEV), eps=1e-5, interleaved=inter)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(d.cpu()[:, (hq + hk) * D:], qkv[:, (hq + hk) * D:])


@pytest.mark.parametrize("T,hq,hk,D,r,inter", CASES + [(4099, 2, 1, 64, 64, False)])
@pytest.mark.parametrize("odd", [False, True])
def test_gradient(T, hq, hk, D, r, inter, odd):
    announce(f"norm_rope_grad {T} {hq} {hk} {D} {r} {inter} odd={odd}")
    qkv, w, cs, pos = _inputs(T, hq, hk, D, r, T + D, odd=odd)
    gr = _inputs(T, hq, hk, D, r, T + D + 1, odd=odd)[0]
    q, k = _views(qkv.to(DEV), hq, hk, D)
    gq, gk = _views(gr.to(DEV), hq, hk, D)
    dq, dk = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, hk, D, dtype=torch.bfloat16, device=DEV)
    dw = [torch.full((D,), 5.0, device=DEV) for _ in range(2)]
    ws = torch.zeros(ar.ar_qk_norm_rope_bwd_workspace(T, hq, hk, D), dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(3):  # one workspace, the same bits each time
        ar.ar_qk_norm_rope_bwd(gq, gk, q, k, w[0].to(DEV), w[1].to(DEV), cs.to(DEV), pos.to(DEV), dq, dk, *dw, ws,
                               eps=1e-5, interleaved=inter)
        got = [x.clone() for x in (dq, dk, *dw)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    xs, gs = _views(qkv, hq, hk, D), _views(gr, hq, hk, D)
    for x, g, wt, dx, dwt, n in zip(xs, gs, w, (dq, dk), dw, "qk"):
        if x.numel():
            want, size, wantw, sizew = R.norm_rope_grad(g, x, wt, cs[pos], 1e-5, inter)
            _close(dx, want, size, 2.0 ** -17, "d" + n)
            off = (dwt.cpu().double() - wantw).abs()
            assert bool((off <= 2.0 ** -16 * sizew + 1e-30).all()), f"d{n}_weight"


def test_definition_of_the_gradient_by_differences():
    """The 64-bit gradient against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(3)
    x, gy = torch.randn(2, 3, 64, generator=g).double(), torch.randn(2, 3, 64, generator=g).double()
    w = 1 + 0.2 * torch.randn(64, generator=g).double()
    a = torch.rand(2, 16, generator=g).double() * 6
    cs = torch.cat([a.cos(), a.sin()], 1)
    dx, _, dw, _ = R.norm_rope_grad(gy, x, w, cs, 1e-5, True)

    def loss(x, w):
        return float((R.norm_rope(x, w, cs, 1e-5, True)[0] * gy).sum())

    for _ in range(8):
        u, uw, e = torch.randn(x.shape, generator=g).double(), torch.randn(64, generator=g).double(), 1e-5
        num = (loss(x + e * u, w + e * uw) - loss(x - e * u, w - e * uw)) / (2 * e)
        assert abs(num - float((dx * u).sum() + (dw * uw).sum())) < 1e-6 * (1 + abs(num))


def test_positions_outside_the_table_give_nan_rows():
    qkv, w, cs, pos = _inputs(4, 2, 1, 128, 128, 5)
    pos = torch.tensor([0, -1, 97, 96])
    q, k = _views(qkv.to(DEV), 2, 1, 128)
    ar.ar_qk_norm_rope(q, k, w[0].to(DEV), w[1].to(DEV), cs.to(DEV), pos.to(DEV))
    nan = torch.isnan(q.float()).all(-1).all(-1).cpu()
    assert nan.tolist() == [False, True, True, False]
    assert not torch.isnan(q.float()[[0, 3]]).any() and bool(torch.isnan(k.float()[1:3]).all())


def test_no_tokens():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    dw = [torch.full((64,), 5.0, device=DEV) for _ in range(2)]
    args = (z(64), z(64), z(9, 64, t=torch.float32), z(0, t=torch.int64))
    ws = torch.zeros(ar.ar_qk_norm_rope_bwd_workspace(0, 2, 1, 64), dtype=torch.uint8, device=DEV)
    ar.ar_qk_norm_rope(z(0, 2, 64), z(0, 1, 64), *args)
    ar.ar_qk_norm_rope_bwd(z(0, 2, 64), z(0, 1, 64), z(0, 2, 64), z(0, 1, 64), *args, z(0, 2, 64), z(0, 1, 64), *dw, ws)
    assert not dw[0].any() and not dw[1].any()
