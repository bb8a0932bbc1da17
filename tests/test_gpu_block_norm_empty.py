"""The gradient of the norms around a block for no tokens: a gate of each token has an
empty gradient, and what all tokens share gets zeros."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [5, 64, 9000])
def test_no_tokens_with_a_gate_for_each(D):
    announce(f"block_norm_grad of no tokens {D}")
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    ws = torch.full((ar.ar_block_norm_bwd_workspace(0, D),), 255, dtype=torch.uint8, device=DEV)
    grads = [torch.full((D,), 5.0, device=DEV) for _ in range(2)]
    ar.ar_block_norm_bwd(z(0, D), z(0, D), z(0, D), z(0, D), z(0, D), z(0, D), ws, post_weight=z(D), gate=z(0, D), pre_weight=z(D), gate_grad=z(0, D),
                         post_grad=grads[0], pre_grad=grads[1])
    assert not any(bool(g.any()) for g in grads)
