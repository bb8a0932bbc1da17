"""GPU parity of the 4-bit cache: every byte written and every value read back
equals the definition's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


def _rows(T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(2 * torch.randn(T, H, 1, generator=g))
    # values on the borders between codes, groups of zeros, tiny and huge groups
    x[0, 0, :32] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 4) * torch.tensor([1.0, -1.0] * 16)
    x[-1, -1, :32] = 0
    if T > 2:
        x[1] *= 1e-38
        x[2] *= 1e37
        x[1, 0, -32:] = torch.tensor([6.99, 7.0] * 16)
        x[2, 0, 32:64] = torch.tensor([3.0e38, -3.3e38] * 16)
    return x.bfloat16()


def _same(o, want):
    """Equal values, NaN where NaN is wanted (a group with an infinity in it)."""
    o = o.cpu().double()
    return torch.equal(torch.isnan(o), torch.isnan(want)) and torch.equal(torch.nan_to_num(o), torch.nan_to_num(want))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,H,page,odd", [(1, 1, 32, False), (5, 2, 32, True), (77, 3, 64, False), (300, 1, 256, True)])
def test_write_and_read(D, T, H, page, odd):
    announce(f"kv4 {D} {T} {H} {page} odd={odd}")
    pages = 2 * -(-T // page) + 1
    k, v = _rows(T, H, D, T + D), _rows(T, H, D, T + D + 1)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T]
    pad = 1 if odd else 0
    both = torch.zeros(T, 2 * H * D + pad, dtype=torch.bfloat16)
    both[:, :2 * H * D] = torch.cat([k, v], 1).reshape(T, -1)
    both = both.to(DEV)
    view = both[:, :2 * H * D].unflatten(1, (2 * H, D))
    cache = torch.full((pages, H, page // 32, 34 * D), 0xA5, dtype=torch.uint8, device=DEV)
    assert cache.numel() == ar.ar_kv4_cache_bytes(pages, H, D, page)
    ar.ar_kv4_write(view[:, :H], view[:, H:], slots.to(DEV), cache, page)
    want = np.full((pages, H, page // 32, 34 * D), 0xA5, dtype=np.uint8)
    kc, kb, vc, vb = (x.copy() for x in R.unpack(want, D))
    p, tile, t = slots.numpy() // page, slots.numpy() % page // 32, slots.numpy() % 32
    for x, codes, scales in ((k, kc, kb), (v, vc, vb)):
        c, b = R.quantise(x)
        codes[p, :, tile, t], scales[p, :, tile, t] = c, b
    assert np.array_equal(cache.cpu().numpy(), R.pack(kc, kb, vc, vb))
    ko, vo = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
    ar.ar_kv4_read(cache, slots.to(DEV), ko, vo, page)
    for x, o in ((k, ko), (v, vo)):
        want = torch.from_numpy(R.values(*R.quantise(x)))
        assert _same(o, want)
    ar.ar_kv4_read(cache, slots.to(DEV), view[:, H:], view[:, :H], page)  # strided, exchanged
    assert _same(view[:, :H], vo.cpu().double()) and _same(view[:, H:], ko.cpu().double())


def test_every_pattern():
    """All bf16 patterns, each beside 31 zeros and beside a largest value."""
    bits = np.arange(65536, dtype=np.uint16)
    x = np.zeros((65536, 1, 64), dtype=np.uint16)
    x[:, 0, 5] = bits
    x[:, 0, 40] = bits
    x[:, 0, 41] = (bits & 0x7F80) + 0x0080 * ((bits & 0x7F80) < 0x7F00)
    k = torch.from_numpy(x.view(np.int16)).view(torch.bfloat16)
    slots = torch.arange(65536)
    cache = torch.zeros(2048, 1, 1, 34 * 64, dtype=torch.uint8, device=DEV)
    ar.ar_kv4_write(k.to(DEV), k.to(DEV), slots.to(DEV), cache, 32)
    ko, vo = torch.empty_like(k, device=DEV), torch.empty_like(k, device=DEV)
    ar.ar_kv4_read(cache, slots.to(DEV), ko, vo, 32)
    want = torch.from_numpy(R.values(*R.quantise(k)))
    assert _same(ko, want) and _same(vo, want)


def test_slots_outside_the_cache():
    D, page = 128, 32
    k = _rows(6, 2, D, 1).to(DEV)
    slots = torch.tensor([-1, 3, 64, 1 << 40, 33, -(1 << 62)], device=DEV)
    cache = torch.zeros(2, 2, 1, 34 * D, dtype=torch.uint8, device=DEV)
    guard = cache.clone()
    ar.ar_kv4_write(k, k, slots, cache, page)
    ar.ar_kv4_write(k[[1, 4]].contiguous(), k[[1, 4]].contiguous(), slots[[1, 4]].contiguous(), guard, page)
    assert torch.equal(cache, guard)
    ko, vo = torch.full_like(k, 9), torch.full_like(k, 9)
    ar.ar_kv4_read(cache, slots, ko, vo, page)
    assert not ko[[0, 2, 3, 5]].any() and not vo[[0, 2, 3, 5]].any()
    want = torch.from_numpy(R.values(*R.quantise(k[[1, 4]].cpu())))
    assert _same(ko[[1, 4]], want) and _same(vo[[1, 4]], want)


def test_groups_that_are_not_finite():
    D = 64
    x = torch.ones(4, 1, D, dtype=torch.bfloat16)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 63] = float("inf"), float("nan"), float("-inf")
    cache = torch.zeros(1, 1, 1, 34 * D, dtype=torch.uint8, device=DEV)
    slots = torch.arange(4, device=DEV)
    ar.ar_kv4_write(x.to(DEV), x.to(DEV), slots, cache, 32)
    ko, vo = torch.empty_like(x, device=DEV), torch.empty_like(x, device=DEV)
    ar.ar_kv4_read(cache, slots, ko, vo, 32)
    want = torch.ones(4, 2, 32, dtype=torch.bool)
    want[0, 0] = want[1, 1] = want[2, 1] = False
    for o in (ko, vo):
        assert torch.equal(~torch.isnan(o.cpu()).reshape(4, 2, 32), want)
        assert bool((o.cpu().reshape(4, 2, 32)[want] == 1).all())
