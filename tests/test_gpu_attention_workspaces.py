"""One workspace of a program's largest call, with guards behind it, used by its
smaller calls: right results, and nothing written past it."""
from __future__ import annotations

import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_kv4_attention import Case
from test_gpu_norm_rope import _inputs, _views

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


def test_gradients_in_the_largest_calls_workspace():
    """Weights' gradients to 2^-16 of their terms' sizes, as in
    test_gpu_norm_rope.py."""
    hq, hk, D = 30, 5, 128
    size = ar.ar_qk_norm_rope_bwd_workspace(4100, hq, hk, D)
    whole = torch.full((size + (1 << 20),), 0x5A, dtype=torch.uint8, device=DEV)
    for T in (4100, 2049, 2048, 1025, 700, 3):
        announce(f"norm_rope_grad workspace {T}")
        qkv, w, cs, pos = _inputs(T, hq, hk, D, 64, T)
        gr = _inputs(T, hq, hk, D, 64, T + 1)[0]
        d = lambda x: x.to(DEV)  # noqa: E731
        (q, k), (gq, gk) = _views(d(qkv), hq, hk, D), _views(d(gr), hq, hk, D)
        dw = [torch.full((D,), 5.0, device=DEV) for _ in range(2)]
        ar.ar_qk_norm_rope_bwd(gq, gk, q, k, d(w[0]), d(w[1]), d(cs), d(pos), gq, gk, *dw, whole[:size], eps=1e-5)
        for x, g, wt, got in zip(_views(qkv, hq, hk, D), _views(gr, hq, hk, D), w, dw):
            _, _, want, sizes = R.norm_rope_grad(g, x, wt, cs[pos], 1e-5, False)
            assert bool(((got.cpu().double() - want).abs() <= 2.0 ** -16 * sizes + 1e-30).all()), T
        assert bool((whole[size:] == 0x5A).all())
