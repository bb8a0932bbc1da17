"""The operators around a block as programs call them: on other streams, from several
threads, in graphs, with one workspace for calls of many sizes, on another GPU."""
from __future__ import annotations

import sys
import threading
import types

import pytest
import torch

from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


class Step:
    """All operators once, on one device."""

    def __init__(self, seed, dev=DEV, T=3, H=320, inner=96, E=12, k=3, P=2, ws=None):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, size=1.0: (size * torch.randn(*s, generator=g)).bfloat16().to(dev)  # noqa: E731
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
        self.parts, self.x, self.dh, self.dz = [n(T, H) for _ in range(P)], n(T, H), n(T, H), n(T, H)
        self.post, self.pre, self.gate = n(H), n(H), n(H)
        self.h, self.z, self.dx, self.dy = z(T, H), z(T, H), z(T, H), z(T, H)
        self.grads = [z(H, t=torch.float32) for _ in range(3)]
        self.w = n(H, H, size=H ** -0.5)
        self.packed, self.back, self.y = z(H // 16, ar.ar_w4_bytes(16, H), t=torch.uint8), z(H, H), z(T, H)
        self.router = n(E, H, size=H ** -0.5)
        self.up, self.down = z(E, inner // 8, ar.ar_w4_bytes(16, H), t=torch.uint8), z(E, H // 16, ar.ar_w4_bytes(16, inner), t=torch.uint8)
        self.raw = [n(2 * inner, H, size=H ** -0.5) for _ in range(E)], [n(H, inner, size=inner ** -0.5) for _ in range(E)]
        self.out, self.choice, self.weight = z(T, H), z(T, k, t=torch.int32), z(T, k, t=torch.float32)
        size = max(ar.ar_block_norm_bwd_workspace(T, H), ar.ar_w4_experts_workspace(T, H, inner, E, k))
        self.ws = z(size, t=torch.uint8) if ws is None else ws
        if dev != DEV:
            torch.cuda.synchronize(dev)

    def run(self, stream=None):
        kw = dict(post_weight=self.post, gate=self.gate, pre_weight=self.pre, stream=stream)
        ar.ar_block_norm(self.parts, self.x, self.h, self.z, **kw)
        ar.ar_block_norm_bwd(self.dh, self.dz, self.parts[0], self.x, self.dx, self.dy, self.ws, gate_grad=self.grads[0], post_grad=self.grads[1],
                             pre_grad=self.grads[2], **kw)
        ar.ar_w4_pack(self.w, self.packed, stream=stream)
        ar.ar_w4_unpack(self.packed, self.back, stream=stream)
        for raw, to in zip(self.raw, (self.up, self.down)):
            for w, p in zip(raw, to):
                ar.ar_w4_pack(w, p, stream=stream)
        ar.ar_w4_linear(self.z, self.packed, self.y, stream=stream)
        ar.ar_w4_experts(self.z, self.router, self.up, self.down, self.out, self.choice, self.weight, self.ws, stream=stream)

    def results(self):
        return [t.clone() for t in (self.h, self.z, self.dx, self.dy, *self.grads, self.back, self.y, self.out, self.choice, self.weight)]


def same(a, b):
    return all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(a, b))


def test_streams():
    announce("block operators on a stream of their own, and on one given")
    s = Step(1)
    s.run()
    want = s.results()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = Step(1)
    torch.cuda.synchronize()
    other.run(stream=side)
    side.synchronize()
    assert same(other.results(), want)
    third = Step(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        third.run()
        got = third.results()
    side.synchronize()
    assert same(got, want)


def test_a_stream_of_another_device_is_refused():
    current = torch.cuda.current_stream()
    far = types.SimpleNamespace(cuda_stream=current.cuda_stream, device_index=current.device_index + 1)
    s = Step(2)
    for call in (lambda: ar.ar_block_norm(s.parts, s.x, s.h, stream=far), lambda: ar.ar_w4_linear(s.x, s.packed, s.y, stream=far),
                 lambda: ar.ar_w4_pack(s.w, s.packed, stream=far)):
        with pytest.raises(ValueError, match="stream"):
            call()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_of_a_device_that_is_not_current():
    announce("block operators on cuda:1 while cuda:0 is current")
    torch.cuda.set_device(0)
    a, b = Step(3), Step(3, "cuda:1")
    a.run()
    b.run()
    torch.cuda.synchronize(0)
    torch.cuda.synchronize(1)
    assert torch.cuda.current_device() == 0 and same(a.results(), b.results())


def test_one_workspace_for_calls_of_many_sizes():
    announce("block operators with one workspace")
    big = dict(T=70, H=512, inner=160, E=40, k=8)
    sizes = [big, dict(T=1, H=64, inner=32, E=1, k=1), dict(T=9, H=320, inner=96, E=12, k=3), dict(T=70, H=512, inner=32, E=40, k=2), big]
    ws = Step(0, **big).ws
    ws.fill_(255)
    for i, size in enumerate(sizes):
        own, shared = Step(i, **size), Step(i, ws=ws, **size)
        own.run()
        shared.run()
        assert same(own.results(), shared.results())


def test_graphs():
    """Captured calls, replayed on other inputs with eager work between."""
    announce("block operators in a graph")
    s, others = Step(4, T=20), [Step(i, T=20) for i in range(5, 9)]
    fields = ("x", "dh", "dz", "post", "pre", "gate", "w", "router")
    want = []
    for o in others:
        o.run()
        want.append(o.results())
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in (0, 3, 1, 2, 0):
        for f in fields:
            getattr(s, f).copy_(getattr(others[i], f))
        for a, b in zip((*s.parts, *s.raw[0], *s.raw[1]), (*others[i].parts, *others[i].raw[0], *others[i].raw[1])):
            a.copy_(b)
        graph.replay()
        assert same(s.results(), want[i])
        others[i].run()
        torch.cuda.synchronize()
        assert same(others[i].results(), want[i])


def test_threads():
    announce("block operators from 6 threads")
    steps = [Step(i, T=5) for i in range(6)]
    want = []
    for s in steps:
        s.run()
        want.append(s.results())
    torch.cuda.synchronize()
    got, failed = [[] for _ in steps], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    steps[i].run()
                    got[i].append(steps[i].results())
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
    assert all(len(g) == 8 and all(same(x, w) for x in g) for g, w in zip(got, want))
