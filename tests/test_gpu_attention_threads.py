"""The attention operators from several threads, each with a stream and buffers of
its own and the threads taking turns as often as the interpreter lets them."""
from __future__ import annotations

import sys
import threading

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        B, self.hq, self.hk, D, self.page, self.n = 3, 8, 2, 128, 64, 700
        self.qkv = torch.randn(B, self.hq + 2 * self.hk, D, generator=g).bfloat16().to(DEV)
        self.raw = self.qkv.clone()
        self.w, self.cs = torch.ones(D, dtype=torch.bfloat16, device=DEV), torch.randn(self.n, D, generator=g).to(DEV)
        self.pos = torch.full((B,), self.n - 1, device=DEV)
        per = -(-self.n // self.page)
        self.table = torch.randperm(B * per, generator=g).reshape(B, per).int().to(DEV)
        self.cache = torch.randint(100, 130, (B * per, self.hk, self.page // 32, 34 * D), generator=g, dtype=torch.uint8).to(DEV)
        self.slots = self.table[:, -1].long() * self.page + (self.n - 1) % self.page
        self.start, self.len = torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.full((B,), self.n, dtype=torch.int32, device=DEV)
        self.out, self.lse = torch.empty(B, self.hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, self.hq, device=DEV)
        self.ws = torch.empty(ar.ar_kv4_attention_workspace(B, B, 1, self.n, self.hq, self.hk, D), dtype=torch.uint8, device=DEV)

    def run(self):
        q, k, v = self.qkv[:, :self.hq], self.qkv[:, self.hq:self.hq + self.hk], self.qkv[:, self.hq + self.hk:]
        self.qkv.copy_(self.raw)
        ar.ar_qk_norm_rope(q, k, self.w, self.w, self.cs, self.pos)
        ar.ar_kv4_write(k, v, self.slots, self.cache, self.page)
        ar.ar_kv4_attention(q, self.cache, self.table, self.start, self.len, self.out, self.lse, self.ws, page_size=self.page,
                            kv_heads=self.hk, max_q=1, max_kv=self.n)
        return self.out.clone(), self.lse.clone()


def test_threads():
    announce("attention operators from 6 threads")
    steps = [Step(i) for i in range(6)]
    want = [s.run() for s in steps]
    torch.cuda.synchronize()
    got, failed = [[] for _ in steps], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [steps[i].run() for _ in range(25)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=work, args=(i,), daemon=True) for i in range(len(steps))]
        for t in threads:
            t.start()
        for t in threads:
            t.join(60)
            assert not t.is_alive()
    finally:
        sys.setswitchinterval(before)
    assert not failed
    for g, w in zip(got, want):
        assert len(g) == 25
        assert all(torch.equal(o, w[0]) and torch.equal(x, w[1]) for o, x in g)
