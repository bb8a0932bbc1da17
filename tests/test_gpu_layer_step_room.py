"""A captured step of the example's layer, replayed until its caches are full and once
more: the last replay looks nothing up past the tables and leaves the caches as they are."""
from __future__ import annotations

import pytest
import torch

from gpu_util import announce
from test_gpu_layer_step import _example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("room", [64, 67])
def test_replays_past_the_room(room):
    announce(f"layer_step replayed past the room {room}")
    E = _example()
    P, B, H = 2, 3, 256
    layer = E.Layer(P, B, H, 2, 1, 64, 64, 8, 2, room)
    g = torch.Generator(device="cuda").manual_seed(5)
    first = torch.randn(B, H, generator=g, device="cuda").bfloat16()
    x, stream = first.clone(), first.clone()

    def start():
        layer.length.fill_(room - 3)
        layer.used = room - 3
        x.copy_(first)
        stream.copy_(first)

    start()
    want = []
    for _ in range(3):
        z = layer.step(x, stream)
        want.append((z.clone(), stream.clone()))
    with pytest.raises(ValueError, match="room"):
        layer.step(x, stream)
    start()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = layer.step(x, stream)
    start()
    for n in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want[n][0]) and torch.equal(stream, want[n][1])
    caches = [r.cache.clone() for r in layer.ranks]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert bool(torch.isnan(z).all()) and bool(torch.isnan(stream).all())
        assert all(torch.equal(a, r.cache) for a, r in zip(caches, layer.ranks))
