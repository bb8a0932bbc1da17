"""The attention operators run on their tensors' GPU, whichever is current."""
from __future__ import annotations

import types

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


def _step(dev, stream=None):
    """All operators once: their outputs."""
    g = torch.Generator().manual_seed(1)
    T, hq, hk, D, page = 5, 4, 2, 64, 32
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    qkv = torch.randn(T, hq + 2 * hk, D, generator=g).bfloat16().to(dev)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    w, cs, at = torch.ones(D, dtype=torch.bfloat16, device=dev), torch.randn(T, D, generator=g).to(dev), torch.arange(T, device=dev)
    qo, ko, dq, dk, ck, cv, out = z(T, hq, D), z(T, hk, D), z(T, hq, D), z(T, hk, D), z(T, hk, D), z(T, hk, D), z(T, hq, D)
    dw, dw2, lse, cache = z(D, t=torch.float32), z(D, t=torch.float32), z(T, hq, t=torch.float32), z(2, hk, 1, 34 * D, t=torch.uint8)
    ws = z(ar.ar_qk_norm_rope_bwd_workspace(T, hq, hk, D), t=torch.uint8)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if dev != DEV:
        torch.cuda.synchronize(dev)
    ar.ar_qk_norm_rope(q, k, w, w, cs, at, qo, ko, stream=stream)
    ar.ar_qk_norm_rope_bwd(q, k, q, k, w, w, cs, at, dq, dk, dw, dw2, ws, stream=stream)
    ar.ar_kv4_write(ko, v, at, cache, page, stream=stream)
    ar.ar_kv4_read(cache, at, ck, cv, page, stream=stream)
    ar.ar_kv4_attention(qo, cache, i32(0, 1)[None], i32(0, T), i32(T), out, lse, ws, page_size=page, kv_heads=hk, max_q=T, max_kv=T,
                        stream=stream)
    torch.cuda.synchronize(dev)
    return [x.cpu() for x in (qo, ko, dq, dk, dw, dw2, ck, cv, out, lse)]


def test_a_stream_of_another_device_is_refused():
    announce("attention operators, a stream of another device")
    current = torch.cuda.current_stream()
    here = types.SimpleNamespace(cuda_stream=current.cuda_stream, device_index=current.device_index)
    other = types.SimpleNamespace(cuda_stream=current.cuda_stream, device_index=current.device_index + 1)
    want = _step(DEV)
    assert all(torch.equal(a, b) for a, b in zip(_step(DEV, here), want))
    assert all(torch.equal(a, b) for a, b in zip(_step(DEV, torch.cuda.current_stream()), want))
    with pytest.raises(ValueError, match="stream"):
        _step(DEV, other)
    assert torch.cuda.current_device() == current.device_index


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_of_a_device_that_is_not_current():
    announce("attention operators on cuda:1 while cuda:0 is current")
    torch.cuda.set_device(0)
    want = _step(DEV)
    got = _step("cuda:1")
    assert torch.cuda.current_device() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
