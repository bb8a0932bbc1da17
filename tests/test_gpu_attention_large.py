"""The kernels that large calls of the attention operators run, each at a call just
past the rule that takes it.  Definitions in 64 bits as in the other files; the
head norms' on the GPU, the cache's by small calls that those files hold to it.

Tolerances are those of test_gpu_norm_rope.py and test_gpu_kv4_attention.py."""
from __future__ import annotations

import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_kv4_attention import Case
from test_gpu_norm_rope import _close, _inputs, _views

pytestmark = pytest.mark.gpu

NORMS = [  # tokens, heads, kv_heads, dim, rotated, interleaved
    (2100, 20, 4, 64, 64, False), (2100, 20, 4, 64, 32, True),       # a wave's steps end on queries and go on with keys
    (2100, 20, 4, 128, 128, False), (2100, 18, 3, 128, 96, True),
    (2100, 20, 4, 256, 256, False), (2100, 19, 5, 256, 128, True),
    (16384, 25, 1, 64, 64, False),                                    # five steps of a wave: more than are in flight
    (8200, 70, 4, 64, 64, False), (8200, 30, 3, 128, 64, True), (8200, 13, 4, 256, 256, False),  # past 128 MiB
    (2100, 0, 24, 128, 128, False), (2100, 24, 0, 64, 64, True)]


@pytest.mark.parametrize("T,hq,hk,D,r,inter", NORMS)
@pytest.mark.parametrize("odd", [False, True])
def test_norms(T, hq, hk, D, r, inter, odd):
    if odd and T > 2100:
        pytest.skip("rows of odd strides take one kernel at all sizes")
    announce(f"large norm_rope {T} {hq} {hk} {D} {r} {inter} odd={odd}")
    qkv, w, cs, pos = _inputs(T, hq, hk, D, r, T + D, odd=odd)
    d = qkv.to(DEV)
    raw = d.clone()
    q, k = _views(d, hq, hk, D)
    qo, ko = torch.full((T, hq, D), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((T, hk, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ww, table, at = [x.to(DEV) for x in w], cs.to(DEV), pos.to(DEV)
    ar.ar_qk_norm_rope(q, k, *ww, table, at, qo, ko, eps=1e-5, interleaved=inter)
    for x, wt, o, n in zip((q, k), ww, (qo, ko), "qk"):
        if o.numel():
            want, size = R.norm_rope(x, wt, table[at], 1e-5, inter)
            _close(o, want.cpu(), size.cpu(), 2.0 ** -18, n)
    ar.ar_qk_norm_rope(q, k, *ww, table, at, eps=1e-5, interleaved=inter)  # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(d[:, (hq + hk) * D:], raw[:, (hq + hk) * D:])


@pytest.mark.parametrize("T,hq,hk,D,r,inter", [(8200, 50, 4, 64, 64, False), (8200, 20, 3, 128, 64, True), (8200, 9, 4, 256, 256, False)])
def test_gradients_past_128_mib(T, hq, hk, D, r, inter):
    announce(f"large norm_rope_grad {T} {hq} {hk} {D} {r} {inter}")
    assert 6 * T * (hq + hk) * D > 128 << 20
    qkv, w, cs, pos = _inputs(T, hq, hk, D, r, T + D)
    gr = _inputs(T, hq, hk, D, r, T + D + 1)[0]
    (q, k), (gq, gk) = _views(qkv.to(DEV), hq, hk, D), _views(gr.to(DEV), hq, hk, D)
    dq, dk = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, hk, D, dtype=torch.bfloat16, device=DEV)
    dw = [torch.full((D,), 5.0, device=DEV) for _ in range(2)]
    ww, table, at = [x.to(DEV) for x in w], cs.to(DEV), pos.to(DEV)
    ws = torch.zeros(ar.ar_qk_norm_rope_bwd_workspace(T, hq, hk, D), dtype=torch.uint8, device=DEV)
    ar.ar_qk_norm_rope_bwd(gq, gk, q, k, *ww, table, at, dq, dk, *dw, ws, eps=1e-5, interleaved=inter)
    for x, g, wt, dx, dwt, n in zip((q, k), (gq, gk), ww, (dq, dk), dw, "qk"):
        want, size, wantw, sizew = R.norm_rope_grad(g, x, wt, table[at], 1e-5, inter)
        _close(dx, want.cpu(), size.cpu(), 2.0 ** -17, "d" + n)
        assert bool(((dwt.double() - wantw).abs() <= 2.0 ** -16 * sizew + 1e-30).all()), f"d{n}_weight"


@pytest.mark.parametrize("T,H,D", [(8203, 2, 64), (8203, 2, 128), (8203, 2, 256), (33001, 4, 64), (16405, 4, 128), (8203, 8, 256)])
@pytest.mark.parametrize("odd", [False, True])
def test_cache(T, H, D, odd):
    """Whole calls against calls of 500 tokens."""
    announce(f"large kv4 {T} {H} {D} odd={odd}")
    assert (T + 7) // 8 * H >= 2048 and (H == 2 or 4 * T * H * D > 32 << 20)
    page, pages, pad = 64, 2 * -(-T // 64) + 1, int(odd)
    g = torch.Generator(device=DEV).manual_seed(T + D)
    store = torch.zeros(T, 2 * H * D + pad, dtype=torch.bfloat16, device=DEV)
    store[:, :2 * H * D] = (torch.randn(T, 2 * H, D, generator=g, device=DEV) *
                            torch.exp(2 * torch.randn(T, 2 * H, 1, generator=g, device=DEV))).reshape(T, -1).bfloat16()
    k, v = store[:, :H * D].unflatten(1, (H, D)), store[:, H * D:2 * H * D].unflatten(1, (H, D))
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
    slots[T // 2] = -1  # outside
    whole, parts = (torch.full((pages, H, page // 32, 34 * D), 0xA5, dtype=torch.uint8, device=DEV) for _ in range(2))
    ar.ar_kv4_write(k, v, slots, whole, page)
    for i in range(0, T, 500):
        ar.ar_kv4_write(k[i:i + 500], v[i:i + 500], slots[i:i + 500], parts, page)
    assert torch.equal(whole, parts)
    want = torch.from_numpy(R.values(*R.quantise(k[T - 100:].cpu())))
    out = torch.full((T, 2 * H * D + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    ko, vo = out[:, :H * D].unflatten(1, (H, D)), out[:, H * D:2 * H * D].unflatten(1, (H, D))
    ar.ar_kv4_read(whole, slots, ko, vo, page)
    kp, vp = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    for i in range(0, T, 500):
        ar.ar_kv4_read(whole, slots[i:i + 500], kp[i:i + 500], vp[i:i + 500], page)
    assert torch.equal(ko, kp) and torch.equal(vo, vp) and not ko[T // 2].any()
    assert torch.equal(ko[T - 100:].cpu().double(), want)
    assert bool((out[:, 2 * H * D:] == 7).all())


ROWS = [(64, 16), (64, 30), (64, 48), (128, 11), (128, 32), (256, 16)]  # dim, rows of a key head: one to three row tiles


@pytest.mark.parametrize("D,rows", ROWS)
def test_many_sequences(D, rows):
    """Row blocks enough for the compute units without ranges: four waves to each."""
    announce(f"many sequences {D} {rows}")
    B, hk = 66, 8
    c = Case([rows] * B, [(37 * b) % 300 for b in range(B)], hk, hk, D, 64, seed=rows)
    c.check(*c.run())


@pytest.mark.parametrize("D,rows", ROWS)
@pytest.mark.parametrize("ranges", [3, 13, 50, 70])
def test_ranges_of_a_long_sequence(D, rows, ranges):
    """Every launch that joins ranges: up to 4, 16, 64 and 256 of them."""
    announce(f"ranges {D} {rows} {ranges}")
    n = ranges * 8 * 32 + 5
    c = Case([1 + (rows - 1) // 8], [n], 8, 1, D, 256, seed=ranges)
    out, lse = c.run()
    c.check(out, lse)
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_ranges_that_stay_empty(D):
    """Ragged lengths in one call of 100 ranges: some sequences have one, one has
    none, and the bound on the lengths is far above all."""
    announce(f"empty ranges {D}")
    c = Case([1, 1, 1], [26000, 301, 0], 4, 1, D, 64)
    c.check(*c.run())
    c.check(*c.run(max_kv=150000))


def test_the_most_ranges():
    announce("256 ranges")
    c = Case([1], [66000], 8, 1, 64, 256)
    c.check(*c.run())
