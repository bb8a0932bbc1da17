"""GPU parity of the mixture-of-experts layer against the 64-bit definitions.

Tolerances.  The experts taken are those of the logits in 64 bits, rounded to
binary32: equal.  Their weights are a softmax of up to 16 in binary32: 2^-20.  The
products are off by 2^-17 of their terms' magnitudes (test_gpu_w4.py), silu by that
times its steepest slope and a few 2^-22 of itself, the result in two bf16 parts
by 2^-17: with the sizes that the definition adds up, 2^-15 of them, and the
rounding of the output, half a step of bf16: 2^-8 of it."""
from __future__ import annotations

import pytest
import torch

import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_w4 import close

pytestmark = pytest.mark.gpu

CASES = [  # tokens, hidden, inner, experts, top_k
    (1, 32, 32, 1, 1), (1, 160, 96, 3, 2), (2, 512, 32, 8, 8), (9, 1056, 128, 37, 4), (16, 256, 160, 16, 1), (17, 96, 288, 16, 6),
    (40, 544, 64, 64, 8), (64, 160, 96, 8, 8), (64, 64, 32, 130, 16), (65, 128, 64, 20, 3), (130, 96, 32, 5, 2), (5, 1024, 64, 512, 8),
    (1, 7168, 64, 32, 8), (33, 64, 544, 4, 1), (3, 2080, 1056, 6, 5), (60, 320, 1024, 48, 8)]


class Layer:
    def __init__(self, T, H, I, E, seed, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.full((T, H + pad), 3.0, dtype=torch.bfloat16)
        self.x[:, :H] = torch.randn(T, H, generator=g).bfloat16()
        self.router = (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16()
        up = [R.random_weights(2 * I, H, g, H ** -0.5) for _ in range(E)]
        down = [R.random_weights(H, I, g, I ** -0.5) for _ in range(E)]
        self.up, self.down = [w for _, w in up], [w for _, w in down]
        self.packed_up, self.packed_down = torch.stack([p for p, _ in up]), torch.stack([p for p, _ in down])
        self.T, self.H, self.I, self.E, self.pad = T, H, I, E, pad

    def run(self, k, scale=1.0):
        out = torch.full((self.T + 2, self.H + self.pad), 7.0, dtype=torch.bfloat16, device=DEV)
        choice = torch.full((self.T + 1, k), -5, dtype=torch.int32, device=DEV)
        weight = torch.full((self.T + 1, k), -5.0, device=DEV)
        n = ar.ar_w4_experts_workspace(self.T, self.H, self.I, self.E, k)
        ws = torch.full((n + 64,), 255, dtype=torch.uint8, device=DEV)  # NaN whatever it is read as
        d = [t.to(DEV) for t in (self.x, self.router, self.packed_up, self.packed_down)]
        ar.ar_w4_experts(d[0][:, :self.H], *d[1:], out[1:-1, :self.H], choice[:-1], weight[:-1], ws[:n], scale=scale)
        assert bool((ws[n:] == 255).all()) and bool((choice[-1] == -5).all()) and bool((weight[-1] == -5).all())
        got = out[1:-1, :self.H].clone()
        out[1:-1, :self.H] = 7.0
        assert bool((out == 7.0).all())
        return got, choice[:-1].cpu(), weight[:-1].cpu()


@pytest.mark.parametrize("T,H,I,E,k", CASES)
@pytest.mark.parametrize("pad", [0, 5])
def test_layer(T, H, I, E, k, pad):
    announce(f"w4_experts {T} {H} {I} {E} {k} pad={pad}")
    layer = Layer(T, H, I, E, T + H + E, pad)
    scale = 1.0 if pad else 2.5
    out, choice, weight = layer.run(k, scale)
    (value, size), c, w = R.experts(layer.x[:, :H], layer.router, layer.up, layer.down, k, scale)
    assert torch.equal(choice.long(), c)
    assert bool(((weight.double() - w).abs() <= 2.0 ** -20 * w).all())
    close(out, value, size, "out", 2.0 ** -15)
    again = layer.run(k, scale)
    assert torch.equal(again[0], out) and torch.equal(again[1], choice) and torch.equal(again[2], weight)


def test_equal_logits_take_the_lower_index():
    announce("w4_experts with equal logits")
    layer = Layer(6, 64, 32, 70, 5)
    layer.router[:] = layer.router[3]
    layer.router[40] *= 2
    layer.router[50] = -layer.router[40]
    _, choice, weight = layer.run(5)
    for t in range(6):
        first, rest = choice[t, 0].item(), choice[t, 1:].tolist()
        assert first in (40, 50) and rest == [0, 1, 2, 3]
        assert weight[t, 1:].unique().numel() == 1


def test_zero_logits_of_either_sign_are_equal():
    announce("w4_experts with zeros")
    layer = Layer(3, 64, 32, 9, 6)
    layer.router[:] = 0
    layer.router[4] = -0.0
    out, choice, weight = layer.run(4)
    assert choice.tolist() == [[0, 1, 2, 3]] * 3 and bool((weight == 0.25).all())
    assert bool(torch.isfinite(out).all())


def test_nan_and_infinities_stay_with_their_tokens():
    announce("w4_experts with NaN")
    layer = Layer(9, 160, 96, 12, 7)
    clean, c, _ = layer.run(3)
    # an expert of NaN weights: the tokens that take it, and no other
    bad = int(c[0, 0])
    layer.packed_down[bad, :, -256:] = 255
    out, choice, _ = layer.run(3)
    takes = (choice == bad).any(1)
    assert torch.equal(choice, c) and 0 < int(takes.sum()) < 9
    assert bool(torch.isnan(out.cpu()[takes]).all()) and torch.equal(out.cpu()[~takes], clean.cpu()[~takes])
    layer = Layer(9, 160, 96, 12, 7)
    layer.x[4, 9], layer.x[6, 0] = float("nan"), float("inf")
    out, choice, weight = layer.run(3)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(out[keep], clean[keep]) and torch.equal(choice[keep], c[keep])
    assert bool(torch.isnan(out[4]).all()) and bool(torch.isnan(weight[4]).all()) and choice[4].tolist() == [0, 1, 2]
    assert bool((choice[6] >= 0).all()) and bool((choice[6] < 12).all()) and len(set(choice[6].tolist())) == 3


def test_no_tokens():
    layer = Layer(1, 64, 32, 2, 1)
    layer.x, layer.T = layer.x[:0], 0
    out, choice, weight = layer.run(1)
    assert out.shape == (0, 64)
