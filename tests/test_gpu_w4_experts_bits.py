"""How many bits the experts' activations keep between the two products.

Units come in pairs whose activations a and a (1 + d) differ by about 2^-13 of
themselves, and an output is the difference of one pair: what is lost of either stays.

Tolerance.  Every product of a unit and the sum of its two terms are exact in
binary32, and so is the weight of a single expert, 1.  An activation is one product
rounded, 2^-24 of it (silu's own error is the same in both and goes with their
difference), and the three parts of the two cancel in sums that are each off by
2^-24 of a at most: 5 x 2^-24 of a in all.  The definition's size is some 6 a: 2^-23
of it is 12 x 2^-24 of a.  The output's rounding, half a step, adds 2^-8 of it."""
from __future__ import annotations

import pytest
import torch

import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_w4 import close

pytestmark = pytest.mark.gpu

ONE = 2  # the code of 1
MINUS = 10


def weights(H, I):
    """Gate and up (2 I, H), and down (H, I), packed and as values: unit j's gate and up see input 0, an odd unit's up
    input 32 as well, 2^-13 of it; output n is the difference of the units 2 p and 2 p + 1, p = n % (I / 2)."""
    unit, n = torch.arange(I), torch.arange(H)
    up, up_scale = torch.zeros(2 * I, H, dtype=torch.uint8), torch.full((2 * I, H // 32), 127, dtype=torch.uint8)
    up[:I, 0] = (1 + unit // 2 % 7).to(torch.uint8)  # 0.5, 1, ... 6: the same in a pair
    up[I:, 0] = ONE
    up[I + 1::2, 32] = ONE
    up_scale[I:, 1] = 127 - 13
    down, down_scale = torch.zeros(H, I, dtype=torch.uint8), torch.full((H, I // 32), 127, dtype=torch.uint8)
    pair = n % (I // 2)
    down[n, 2 * pair], down[n, 2 * pair + 1] = ONE, MINUS
    out = []
    for code, scale in ((up, up_scale), (down, down_scale)):
        packed = R.pack(code.numpy(), scale.numpy())
        out.append((torch.from_numpy(packed), R.values(packed, *code.shape)))
    return out


# tokens, hidden, inner, experts: products and sums at once with one and two tiles, of more tokens, and apart, with one
# and two tiles to a wave and one and two groups of tokens
@pytest.mark.parametrize("T,H,I,E", [(1, 64, 32, 1), (5, 96, 160, 1), (3, 4160, 96, 1), (8, 64, 544, 2), (20, 64, 96, 2), (64, 160, 288, 1), (64, 64, 2080, 1),
                                     (64, 96, 800, 16), (64, 8192, 800, 16), (64, 16384, 1056, 8), (9, 64, 17440, 2)])
def test_activations_keep_binary32(T, H, I, E):
    announce(f"w4_experts bits {T} {H} {I} {E}")
    g = torch.Generator().manual_seed(T + H + I)
    (up, up_value), (down, down_value) = weights(H, I)
    x = torch.randn(T, H, generator=g).bfloat16()
    x[:, 0] = 1 + torch.rand(T, generator=g).bfloat16()
    x[:, 32] = (1 + torch.rand(T, generator=g)).bfloat16()
    router = (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16()
    out, choice = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, 1, dtype=torch.int32, device=DEV)
    weight, ws = torch.empty(T, 1, device=DEV), torch.full((ar.ar_w4_experts_workspace(T, H, I, E, 1),), 255, dtype=torch.uint8, device=DEV)
    d_up, d_down = up.to(DEV).repeat(E, 1, 1), down.to(DEV).repeat(E, 1, 1)
    ar.ar_w4_experts(x.to(DEV), router.to(DEV), d_up, d_down, out, choice, weight, ws)
    (value, size), c, _ = R.experts(x, router, [up_value] * E, [down_value] * E, 1, 1.0)
    assert torch.equal(choice.cpu().long(), c) and bool((weight == 1).all())
    assert bool((value.abs() < 2.0 ** -11 * size).all()) and bool((value != 0).all())
    close(out, value, size, "out", 2.0 ** -23)


@pytest.mark.parametrize("T", [1, 6, 20])
def test_activations_beyond_bf16(T):
    """Activations between the largest bf16, 2^128 - 2^120, and the largest binary32: no part of one is infinite."""
    announce(f"w4_experts large activations {T}")
    H, I, E = 64, 32, 1
    up, up_scale = torch.zeros(2 * I, H, dtype=torch.uint8), torch.full((2 * I, H // 32), 127, dtype=torch.uint8)
    up[:I, 0], up[I:, 32], up[I:, 33] = ONE, ONE, ONE
    up_scale[:I, 0] = 127 + 10
    down, down_scale = torch.zeros(H, I, dtype=torch.uint8), torch.full((H, I // 32), 127 - 20, dtype=torch.uint8)
    down[:, 3] = ONE
    packed = [R.pack(c.numpy(), s.numpy()) for c, s in ((up, up_scale), (down, down_scale))]
    value = [R.values(p, *c.shape) for p, c in zip(packed, (up, down))]
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    x[:, 0] = 1.0
    # silu(2^10) = 2^10: 2^10 (2^118 - 2^110 + 3 x 2^108) is three quarters of a step above the largest bf16
    x[:, 32], x[:, 33] = 2.0 ** 118 - 2.0 ** 110, 3 * 2.0 ** 108
    router = torch.zeros(E, H, dtype=torch.bfloat16)
    out, choice = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, 1, dtype=torch.int32, device=DEV)
    weight, ws = torch.empty(T, 1, device=DEV), torch.empty(ar.ar_w4_experts_workspace(T, H, I, E, 1), dtype=torch.uint8, device=DEV)
    ar.ar_w4_experts(x.to(DEV), router.to(DEV), torch.from_numpy(packed[0]).to(DEV)[None], torch.from_numpy(packed[1]).to(DEV)[None], out, choice, weight, ws)
    (want, size), _, _ = R.experts(x, router, [value[0]], [value[1]], 1, 1.0)
    assert bool((want > 2.0 ** 107).all()) and bool((want < 2.0 ** 109).all())
    close(out, want, size, "out", 2.0 ** -20)
