"""CPU tests of calls of the operators around a block with no tokens: they pass the
same checks as others, and are refused for nothing that is there but empty."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _bwd(tokens, **kw):
    a = dict(h_grad=_bf(tokens, 64), z_grad=_bf(tokens, 64), y=_bf(tokens, 64), x=_bf(tokens, 64), dx=_bf(tokens, 64), dy=_bf(tokens, 64),
             workspace=torch.zeros(ar.ar_block_norm_bwd_workspace(tokens, 64), dtype=torch.uint8), post_weight=_bf(64), pre_weight=_bf(64),
             post_grad=torch.zeros(64), pre_grad=torch.zeros(64), stream=0)
    a.update(kw)
    ar.ar_block_norm_bwd(**a)


@pytest.mark.parametrize("tokens", [0, 1, 4])
@pytest.mark.parametrize("shared", [False, True])
def test_a_gate_of_any_number_of_tokens_has_a_gradient(tokens, shared):
    gate, grad = (_bf(64), torch.zeros(64)) if shared else (_bf(tokens, 64), _bf(tokens, 64))
    with pytest.raises(TypeError, match="CUDA"):  # all fits, but nothing is on a GPU
        _bwd(tokens, gate=gate, gate_grad=grad)
    with pytest.raises(ValueError, match="no gate"):
        _bwd(tokens, gate=None, gate_grad=grad)
    with pytest.raises(ValueError, match="gate_grad: (shape|torch)"):
        _bwd(tokens, gate=gate, gate_grad=_bf(tokens, 64) if shared else torch.zeros(64))


@pytest.mark.parametrize("call", [
    lambda z: ar.ar_block_norm([z, z], z, z, _bf(0, 64), post_weight=_bf(64), gate=_bf(0, 64), pre_weight=_bf(64), stream=0),
    lambda z: ar.ar_w4_linear(z, torch.zeros(1, ar.ar_w4_bytes(16, 64), dtype=torch.uint8), _bf(0, 5), stream=0),
    lambda z: ar.ar_w4_experts(z, _bf(3, 64), torch.zeros(3, 4, ar.ar_w4_bytes(16, 64), dtype=torch.uint8), torch.zeros(3, 4, ar.ar_w4_bytes(16, 32), dtype=torch.uint8),
                               _bf(0, 64), torch.zeros(0, 2, dtype=torch.int32), torch.zeros(0, 2),
                               torch.zeros(ar.ar_w4_experts_workspace(0, 64, 32, 3, 2), dtype=torch.uint8), stream=0)])
def test_no_tokens_pass_the_binding(call):
    with pytest.raises(TypeError, match="CUDA"):
        call(_bf(0, 64))
