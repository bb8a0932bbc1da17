"""Gradients of what all tokens share, for many tokens.

Tolerance.  A term is off by 2^-17 of its size (test_gpu_block_norm.py).  Added up one
after another in binary32, with 2^-24 of the terms so far at each addition, are at
most 96 terms, four such sums beyond 8192 channels, sixteen of those and sixteen again:
95 + 3 + 15 + 15 = 128 times 2^-24, 2^-17 of the terms' sizes; between those it is 64
bits.  2^-16 in all.  Equal terms, whose roundings all go one way, are the worst case."""
from __future__ import annotations

import pytest
import torch

import block_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_block_norm import EPS, close

pytestmark = pytest.mark.gpu


def call(t, T, D, post, gate, pre, scale=1.0, gate_rows=False):
    """dx, dy and the sums, in a workspace of exactly the size asked for, between guards."""
    size, guard = ar.ar_block_norm_bwd_workspace(T, D), 1 << 20
    ws = torch.full((size + 2 * guard,), 255, dtype=torch.uint8, device=DEV)
    dx, dy = torch.empty(T, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    grads = {"gate": torch.full((D,), 5.0, device=DEV) if gate is not None else None, "post": torch.full((D,), 5.0, device=DEV) if post is not None else None,
             "pre": torch.full((D,), 5.0, device=DEV) if pre is not None else None}
    ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], t["y"], t["x"], dx, dy, ws[guard:guard + size], post_weight=post, gate=gate, pre_weight=pre,
                         gate_grad=grads["gate"], post_grad=grads["post"], pre_grad=grads["pre"], residual_scale=scale, eps=EPS)
    assert bool((ws[:guard] == 255).all()) and bool((ws[guard + size:] == 255).all())
    return dx, dy, grads


@pytest.mark.parametrize("T,D,norms", [(1 << 22, 8, False), (1 << 22, 8, True), (1 << 22, 5, False), (2100000, 264, False), (1000001, 520, True), (400000, 5120, False),
                                       (300000, 7168, True), (262143, 8200, False), (262144, 8200, True), (150000, 16384, True)])
def test_equal_tokens(T, D, norms):
    announce(f"block_norm_grad of equal tokens {T} {D} {norms}")
    g = torch.Generator().manual_seed(D)
    # products whose sums of 2^8 to 2^12 terms all round downwards: 1.2109 x 1.6484 and the like
    pairs = torch.tensor([(27, 83), (13, 106), (25, 84), (31, 76), (83, 27), (106, 13), (84, 25), (76, 31)])[torch.arange(D) % 8]
    row = {"h_grad": (1 + pairs[:, 0] / 128).bfloat16()[None], "y": (1 + pairs[:, 1] / 128).bfloat16()[None], "x": torch.randn(1, D, generator=g).bfloat16(), "z_grad": None}
    post = pre = None
    if norms:
        post, pre, row["z_grad"] = torch.ones(D).bfloat16(), torch.ones(D).bfloat16(), (1 + torch.rand(1, D, generator=g)).bfloat16()
    gate = torch.ones(D).bfloat16()
    t = {k: None if v is None else v.to(DEV).expand(T, D) for k, v in row.items()}
    d = lambda v: None if v is None else v.to(DEV)  # noqa: E731
    dx, dy, grads = call(t, T, D, d(post), d(gate), d(pre))
    want = R.block_norm_grad(row["h_grad"], row["z_grad"], row["y"], row["x"], post, gate, pre, 1.0, EPS)
    for k, v in grads.items():
        if v is not None:
            close(v, (T * want[k][0], T * want[k][1]), 2.0 ** -16, k)
    for got, k in ((dx, "dx"), (dy, "dy")):
        close(got[:1], want[k], 2.0 ** -17, k)
        assert bool((got == got[:1]).all())


@pytest.mark.parametrize("T,D", [(24576, 1024), (98305, 1025), (40001, 100), (98304, 7), (98305, 264), (262145, 64), (24577, 4104), (33025, 6152), (12289, 8200), (40003, 8200),
                                 (66049, 2056)])
def test_chains_of_every_length(T, D):
    """Workgroups with one chain of tokens or several, some of them one less than others."""
    announce(f"block_norm_grad chains {T} {D}")
    g = torch.Generator(device=DEV).manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    t = {k: n(T, D) for k in ("h_grad", "z_grad", "y", "x")}
    post, gate, pre = n(D), n(D), n(D)
    dx, dy, grads = call(t, T, D, post, gate, pre, 0.75)
    sums = {}
    step = max(1, (1 << 25) // D)
    for at in range(0, T, step):
        r = slice(at, at + step)
        w = R.block_norm_grad(t["h_grad"][r], t["z_grad"][r], t["y"][r], t["x"][r], post, gate, pre, 0.75, EPS)
        for got, k in ((dx, "dx"), (dy, "dy")):
            close(got[r], tuple(v.cpu() for v in w[k]), 2.0 ** -17, k)
        for k in grads:
            sums[k] = tuple(a + b for a, b in zip(sums[k], w[k])) if k in sums else w[k]
    for k, v in grads.items():
        close(v, tuple(a.cpu() for a in sums[k]), 2.0 ** -16, k)
