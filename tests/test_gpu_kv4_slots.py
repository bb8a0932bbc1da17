"""A slot named twice in one write: each byte is either token's, and no other slot
is touched."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,T", [(64, 200), (128, 2000), (256, 70)])
def test_a_slot_named_twice(D, T):
    announce(f"kv4 twice {D} {T}")
    H, page, pages = 2, 64, 2 * -(-T // 64)
    g = torch.Generator().manual_seed(D)
    k, v = torch.randn(T, H, D, generator=g).bfloat16(), 8 * torch.randn(T, H, D, generator=g).bfloat16()
    slots = torch.randperm(pages * page, generator=g)[:T]
    first, second = 3, T - 2  # and two neighbours
    slots[second], slots[11] = slots[first], slots[10]
    cache = torch.full((pages, H, page // 32, 34 * D), 0xA5, dtype=torch.uint8, device=DEV)
    ar.ar_kv4_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache, page)
    got = R.unpack(cache.cpu().numpy(), D)
    want = [x.copy() for x in R.unpack(np.full(cache.shape, 0xA5, dtype=np.uint8), D)]
    other = [x.copy() for x in want]

    def put(to, i):
        s = int(slots[i])
        for x, (c, b) in ((k, (0, 1)), (v, (2, 3))):
            to[c][s // page, :, s % page // 32, s % 32], to[b][s // page, :, s % page // 32, s % 32] = R.quantise(x[i])

    for i in range(T):
        put(want, i)
        put(other, i)
    put(other, first)
    put(other, 10)
    for a, b, c in zip(got, want, other):
        assert np.array_equal(a[b == c], b[b == c])  # every slot but the two
        assert ((a == b) | (a == c)).all()
