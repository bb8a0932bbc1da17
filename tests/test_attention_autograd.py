"""CPU tests: the attention operators' calls record nothing for autograd, and say
so where a gradient would be lost.  Nothing here reaches a GPU: tensors that pass
every check are refused for lying on the CPU (TypeError)."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def _calls():
    """(call, its floating-point tensors) of every operator."""
    D, T = 64, 4
    i32 = torch.int32
    norm = [_bf(T, 8, D), _bf(T, 1, D), _bf(D), _bf(D), torch.zeros(9, D), torch.zeros(T, dtype=torch.int64)]
    yield (lambda: ar.ar_qk_norm_rope(*norm, stream=0)), norm[:5]
    dw = [torch.zeros(D), torch.zeros(D)]
    bwd = [_bf(T, 8, D), _bf(T, 1, D)]
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    yield (lambda: ar.ar_qk_norm_rope_bwd(*bwd, *norm, *bwd, *dw, ws, stream=0)), [*bwd, *norm[:5], *dw]
    kv, slots = [_bf(T, 2, D), _bf(T, 2, D)], torch.zeros(T, dtype=torch.int64)
    cache = torch.zeros(3, 2, 2, 34 * D, dtype=torch.uint8)
    yield (lambda: ar.ar_kv4_write(*kv, slots, cache, 64, stream=0)), kv
    yield (lambda: ar.ar_kv4_read(cache, slots, *kv, 64, stream=0)), kv
    q, out, lse = _bf(T, 8, D), _bf(T, 8, D), torch.zeros(T, 8)
    yield (lambda: ar.ar_kv4_attention(q, cache, torch.zeros(1, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), out,
                                       lse, ws, page_size=64, kv_heads=2, max_q=4, max_kv=100, stream=0)), [q, out, lse]


def test_a_gradient_that_would_be_lost_is_refused():
    for call, tensors in _calls():
        with pytest.raises(TypeError, match="CUDA"):
            call()
        for t in tensors:
            t.requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                call()
            with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):
                call()
            t.requires_grad_(False)


def test_inside_an_autograd_function():
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, call, q):
            with pytest.raises(TypeError, match="CUDA"):  # all checks but the last are passed
                call()
            return q.clone()

    call, tensors = next(_calls())
    tensors[0].requires_grad_()
    Norm.apply(call, tensors[0])
