"""Gradients of the norms around a block for rows with infinities and NaN: what the
definition leaves finite stays finite.

Without a norm before the next block dx and dy do not depend on x, and without one
after this block dy does not depend on y: only the sums over tokens that have such a
factor, and the rows of norms that see it, may lose their value.

Tolerances are those of test_gpu_block_norm.py, with the sizes of the same rows
without their infinities and NaN; where the definition is infinite or NaN the result is
the same infinity or NaN."""
from __future__ import annotations

import pytest
import torch

import block_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_block_norm import BF, EPS, dev, make

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(got, value, size, rel, what):
    got = got.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(value)), f"{what}: NaN in other places, {int(torch.isnan(got).sum())} for {int(torch.isnan(value).sum())}"
    inf = torch.isinf(value)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], value[inf]), f"{what}: infinities"
    ok = torch.isfinite(value)
    off, tol = (got - value)[ok].abs(), (BF * value.abs() + rel * size + 1e-30)[ok]
    assert bool((off <= tol).all()), f"{what}: {float((off / tol).max())} times the tolerance"


@pytest.mark.parametrize("T,D", [(6, 5), (6, 264), (40, 1029), (300, 520), (5, 7000), (6, 8200), (40, 16383)])
@pytest.mark.parametrize("post,pre", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("gate", ["none", "shared", "token"])
@pytest.mark.parametrize("where", ["x", "y", "both"])
def test_what_does_not_depend_on_it_stays(T, D, post, pre, gate, where):
    announce(f"block_norm_grad not finite {T} {D} {post} {pre} {gate} {where}")
    s = make(T, D, 1, post, gate, pre, T + D)
    s["parts"][0][s["parts"][0] == 0] = 0.5  # a row of zeros: infinity in it is the only reason to lose a value
    s["y"] = s.pop("parts")[0]
    clean = {k: s[k].clone() for k in ("x", "y")}
    for k in ("x", "y"):
        if where in (k, "both"):
            s[k][1, D - 1], s[k][3, 0], s[k][4, D // 2] = INF, NAN, -INF
    t = {k: dev(v, D) for k, v in s.items()}
    dx, dy = torch.empty(T, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    grads = {"post": torch.empty(D, device=DEV) if post else None, "pre": torch.empty(D, device=DEV) if pre else None,
             "gate": {"none": None, "shared": torch.empty(D, device=DEV), "token": torch.empty_like(dx)}[gate]}
    ws = torch.full((ar.ar_block_norm_bwd_workspace(T, D),), 255, dtype=torch.uint8, device=DEV)
    ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], t["y"], t["x"], dx, dy, ws, post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                         gate_grad=grads["gate"], post_grad=grads["post"], pre_grad=grads["pre"], residual_scale=0.75, eps=EPS)
    args = (s["post"], s["gate"], s["pre"], 0.75, EPS)
    want = R.block_norm_grad(s["h_grad"], s["z_grad"], s["y"], s["x"], *args)
    sizes = R.block_norm_grad(s["h_grad"], s["z_grad"], clean["y"], clean["x"], *args)
    if not pre:
        assert bool(torch.isfinite(want["dx"][0]).all())
        if where == "x" or not post:
            assert bool(torch.isfinite(want["dy"][0]).all())
    for got, k in ((dx, "dx"), (dy, "dy"), *((v, k) for k, v in grads.items() if v is not None)):
        same(got, want[k][0], sizes[k][1], 2.0 ** -17 if got.dim() > 1 else 2.0 ** -16, k)


@pytest.mark.parametrize("D", [9, 12, 16, 1029, 7001, 8203, 16383])
@pytest.mark.parametrize("post,gate,pre", [(True, "shared", False), (True, "token", True), (True, "none", True), (False, "shared", True)])
def test_an_infinite_weight_counts_once(D, post, gate, pre):
    """An infinity in a gate or a weight, in a channel of the last eight of a row of no round size: the sums that it
    enters are infinite, and NaN only where the definition is."""
    T = 6
    announce(f"block_norm_grad infinite weights {D} {post} {gate} {pre}")
    clean = make(T, D, 1, post, gate, pre, D)
    clean["parts"][0][clean["parts"][0] == 0] = 0.5
    for name in ("post", "gate", "pre"):
        if clean[name] is None:
            continue
        s = {**clean, name: clean[name].clone()}
        s[name][..., D - 6] = INF
        t = {k: dev(v, D) for k, v in s.items() if k != "parts"}
        dx, dy = torch.empty(T, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
        ws = torch.full((ar.ar_block_norm_bwd_workspace(T, D),), 255, dtype=torch.uint8, device=DEV)
        ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], dev(s["parts"][0], D), t["x"], dx, dy, ws, post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                             residual_scale=0.75, eps=EPS)
        want = R.block_norm_grad(s["h_grad"], s["z_grad"], s["parts"][0], s["x"], s["post"], s["gate"], s["pre"], 0.75, EPS)
        sizes = R.block_norm_grad(s["h_grad"], s["z_grad"], s["parts"][0], s["x"], clean["post"], clean["gate"], clean["pre"], 0.75, EPS)
        same(dx, want["dx"][0], sizes["dx"][1], 2.0 ** -17, f"dx of {name}")
        same(dy, want["dy"][0], sizes["dy"][1], 2.0 ** -17, f"dy of {name}")
