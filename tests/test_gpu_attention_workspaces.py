"""One workspace of a program's largest call, with guards behind it, used by its
smaller calls: right results, and nothing written past it."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,hk,D", [(8, 1, 128), (9, 3, 64), (2, 2, 256)])
def test_attention_in_the_largest_calls_workspace(heads, hk, D):
    announce(f"kv4 workspace {heads} {hk} {D}")
    size = ar.ar_kv4_attention_workspace(600, 600, 40, 9000, heads, hk, D)
    whole = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    for qlens, kvlens in (([1], [9000]), ([1] * 3, [9000, 8100, 33]), ([1] * 17, [600] * 17), ([1] * 65, [1030] * 65),
                          ([40], [9000]), ([3, 40], [2100, 1999])):
        c = Case(qlens, kvlens, heads, hk, D, 64)
        c.check(*c.run(whole[:size]))
        assert bool((whole[size:] == 0x5A).all())
