"""The mixture-of-experts layer where all tokens take the same few experts out of many:
an expert's columns are taken in several turns by both products, over several chunks.
The experts that no token takes hold NaN.  Tolerances are those of
test_gpu_w4_experts.py: a sum of the first product has up to 36 instructions one after
another on each of eight waves, of the second 72, below 2^-17 of the terms."""
from __future__ import annotations

import pytest
import torch

import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_w4 import close

pytestmark = pytest.mark.gpu


def run(x, router, up, down, I, E, k):
    T, H = x.shape
    out, choice = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    weight, size = torch.empty(T, k, device=DEV), ar.ar_w4_experts_workspace(T, H, I, E, k)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device=DEV)
    ar.ar_w4_experts(x.to(DEV), router.to(DEV), up, down, out[:-1], choice, weight, ws[:size])
    assert bool((out[-1] == 7.0).all()) and bool((ws[size:] == 255).all())
    return out[:-1], choice.cpu().long(), weight.cpu()


def layer(H, I, E, taken, g):
    """Packed weights of all experts on the GPU, and the values of those taken."""
    up = torch.full((E, I // 8, R.tile_bytes(H)), 255, dtype=torch.uint8, device=DEV)
    down = torch.full((E, H // 16, R.tile_bytes(I)), 255, dtype=torch.uint8, device=DEV)
    values = [None] * E, [None] * E
    for e in taken:
        p, values[0][e] = R.random_weights(2 * I, H, g, H ** -0.5)
        up[e] = p.to(DEV)
        p, values[1][e] = R.random_weights(H, I, g, I ** -0.5)
        down[e] = p.to(DEV)
    return up, down, values


@pytest.mark.parametrize("T,H,I,E,k", [
    # one group at a time, inner sizes past a block of chunks, one tile to a wave and two
    (9, 160, 2208, 16, 3), (17, 416, 2208, 24, 4), (33, 672, 2080, 40, 4), (64, 672, 2208, 64, 5), (33, 2048, 2080, 64, 5), (64, 2048, 1056, 64, 5),
    # one tile of gate and up, of 17, 18 and 19 chunks
    (17, 2176, 992, 16, 1), (33, 2208, 992, 16, 1), (64, 2336, 992, 16, 1), (64, 64, 800, 20, 1),
    # workgroups that take tiles in turn
    (64, 512, 1056, 64, 5), (64, 96, 1056, 128, 5),
    # two groups at a time
    (64, 160, 2208, 8, 3), (33, 416, 1184, 6, 2), (64, 8192, 544, 16, 8), (9, 96, 2208, 4, 3),
    # products and sums at once
    (5, 1056, 160, 64, 8), (5, 4192, 96, 16, 3), (33, 160, 96, 4, 2), (64, 288, 64, 10, 3), (6, 2080, 96, 30, 3), (64, 4192, 32, 12, 2),
    # more tokens than a pass
    (130, 416, 1184, 16, 2)])
def test_the_same_experts_for_all(T, H, I, E, k):
    announce(f"w4_experts skew {T} {H} {I} {E} {k}")
    g = torch.Generator().manual_seed(T + H + I + E)
    taken = sorted(set([0, E - 1] + torch.randperm(E, generator=g).tolist()), key=lambda e: e not in (0, E - 1))[:k]
    up, down, values = layer(H, I, E, taken, g)
    x, router = torch.randn(T, H, generator=g).bfloat16(), (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16()
    x[:, 1] = 2.0
    router[taken, 1] = (10 + torch.rand(k, generator=g)).bfloat16()
    out, choice, weight = run(x, router, up, down, I, E, k)
    (value, size), c, w = R.experts(x, router, *values, k, 1.0)
    assert set(c.unique().tolist()) == set(taken)
    assert torch.equal(choice, c) and bool(((weight.double() - w).abs() <= 2.0 ** -20 * w).all())
    close(out, value, size, "out", 2.0 ** -15)


@pytest.mark.parametrize("T,H,I,E,k", [(20, 96, 2208, 12, 4), (7, 1056, 96, 33, 5), (64, 160, 96, 70, 3), (3, 2080, 64, 17, 8), (1, 544, 32, 70, 5)])
def test_equal_logits(T, H, I, E, k):
    """Experts that are alike to the router: all tokens take the first ones, each by the same weight."""
    announce(f"w4_experts skew, equal logits {T} {H} {I} {E} {k}")
    g = torch.Generator().manual_seed(T)
    up, down, values = layer(H, I, E, range(k), g)
    x, row = torch.randn(T, H, generator=g).bfloat16(), (torch.randn(1, H, generator=g) * H ** -0.5).bfloat16()
    out, choice, weight = run(x, row.expand(E, H).contiguous(), up, down, I, E, k)
    (value, size), c, _ = R.experts(x, row.expand(E, H), *values, k, 1.0)
    assert torch.equal(choice, torch.arange(k).expand(T, k)) and torch.equal(choice, c)
    assert bool(((weight.double() - 1 / k).abs() <= 2.0 ** -20 / k).all())
    close(out, value, size, "out", 2.0 ** -15)
