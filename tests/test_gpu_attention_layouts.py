"""The attention operators on arrays that lie between each other: queries, keys and
values of each head side by side, and head after head.  Written in place, they
give the bits that arrays of their own give, and touch nothing beside them."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu

LAYOUTS = {  # (tokens, heads, 4, dim) as it lies in memory: queries, keys, values, something else
    "token, head, part": (0, 1, 2, 3), "token, part, head": (0, 2, 1, 3), "head, token, part": (1, 0, 2, 3),
    "part, head, token": (2, 1, 0, 3), "head, part, token": (1, 2, 0, 3)}


def _laid(x, order):
    """x's values with that order of the axes in memory, x's own order of the axes to index them."""
    back = [order.index(i) for i in range(4)]
    return x.permute(order).contiguous().to(DEV).permute(back)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D", [(1, 3, 64), (5, 1, 64), (37, 6, 128), (8, 2, 256)])
def test_arrays_between_each_other(layout, T, H, D):
    announce(f"layouts {layout} {T} {H} {D}")
    order = LAYOUTS[layout]
    g = torch.Generator().manual_seed(T + D)
    x, gr = torch.randn(T, H, 4, D, generator=g).bfloat16(), torch.randn(T, H, 4, D, generator=g).bfloat16()
    w = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV) for _ in range(2)]
    cs, pos = torch.randn(50, D, generator=g).to(DEV), torch.randint(0, 50, (T,), generator=g).to(DEV)
    own = [x[:, :, i].contiguous().to(DEV) for i in range(4)]
    grads = [gr[:, :, i].contiguous().to(DEV) for i in range(4)]
    dw = [torch.empty(D, device=DEV) for _ in range(4)]
    ws = torch.empty(ar.ar_qk_norm_rope_bwd_workspace(T, H, H, D), dtype=torch.uint8, device=DEV)

    laid, laid_grads = _laid(x, order), _laid(gr, order)
    ar.ar_qk_norm_rope_bwd(grads[0], grads[1], own[0], own[1], *w, cs, pos, grads[0], grads[1], dw[0], dw[1], ws)
    ar.ar_qk_norm_rope_bwd(laid_grads[:, :, 0], laid_grads[:, :, 1], laid[:, :, 0], laid[:, :, 1], *w, cs, pos, laid_grads[:, :, 0],
                           laid_grads[:, :, 1], dw[2], dw[3], ws)
    assert all(torch.equal(laid_grads[:, :, i], grads[i]) for i in range(4))
    assert torch.equal(dw[0], dw[2]) and torch.equal(dw[1], dw[3])

    ar.ar_qk_norm_rope(own[0], own[1], *w, cs, pos)
    ar.ar_qk_norm_rope(laid[:, :, 0], laid[:, :, 1], *w, cs, pos)
    assert all(torch.equal(laid[:, :, i], own[i]) for i in range(4))

    slots = torch.randperm(64, generator=g)[:T].to(DEV)
    caches = [torch.zeros(2, H, 1, 34 * D, dtype=torch.uint8, device=DEV) for _ in range(2)]
    ar.ar_kv4_write(own[1], own[2], slots, caches[0], 32)
    ar.ar_kv4_write(laid[:, :, 1], laid[:, :, 2], slots, caches[1], 32)
    assert torch.equal(*caches)
    ar.ar_kv4_read(caches[0], slots, own[1], own[2], 32)
    ar.ar_kv4_read(caches[1], slots, laid[:, :, 1], laid[:, :, 2], 32)
    assert all(torch.equal(laid[:, :, i], own[i]) for i in range(4))
