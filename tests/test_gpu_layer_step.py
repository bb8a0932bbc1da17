"""The example's decode steps of a whole layer, all ranks together: each operator's
result against the 64-bit definition of what it was given.

Tolerances are those of the operators' own tests.  The norms, the cache and the
attention over it between the first product and the output projection are held by
test_gpu_decode_share.py; here they have to give numbers of the right size."""
from __future__ import annotations

import importlib.util
import pathlib

import pytest
import torch

import block_ref as N
import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import announce
from test_gpu_block_norm import close as close_norm
from test_gpu_w4 import close

pytestmark = pytest.mark.gpu


def _example():
    path = pathlib.Path(__file__).resolve().parents[1] / "examples" / "layer_step.py"
    spec = importlib.util.spec_from_file_location("layer_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("P,B", [(1, 1), (3, 5), (2, 18)])
def test_steps_of_all_ranks(P, B):
    announce(f"layer_step {P} ranks, {B} sequences")
    E = _example()
    H, hq, hk, D, inner, experts, top_k = 320, 2, 1, 64, 96, 10, 3
    layer = E.Layer(P, B, H, hq, hk, D, inner, experts, top_k, 3)
    g = torch.Generator(device="cuda").manual_seed(2)
    stream = torch.randn(B, H, generator=g, device="cuda").bfloat16()
    x = torch.randn(B, H, generator=g, device="cuda").bfloat16()
    values = [dict(out=R.values(r.out_weight.cpu().numpy(), H, hq * D),
                   up=[R.values(w.cpu().numpy(), 2 * inner, H) for w in r.gate_up], down=[R.values(w.cpu().numpy(), H, inner) for w in r.down])
              for r in layer.ranks]
    seen = []
    plain = layer.join

    def join(half, s):
        before = [r.partial.cpu() for r in layer.ranks], s.cpu(), [r.attended.cpu() for r in layer.ranks]
        z = plain(half, s)
        seen.append((half, *before, s.cpu(), z.cpu()))
        return z

    layer.join = join
    for step in range(3):
        seen.clear()
        x = layer.step(x, stream).clone()
        for half, parts, h_in, attended, h_out, z in seen:
            want = N.block_norm(parts, h_in, layer.post[half].cpu(), layer.gate[half].cpu(), layer.pre[1 - half].cpu(), 1.0, 1e-6)
            close_norm(h_out, want[0], 2.0 ** -18, "stream")
            close_norm(z, want[1], 2.0 ** -18, "input")
            for r in range(P):
                if half == 0:
                    assert bool(torch.isfinite(attended[r]).all()) and 0 < float(attended[r].float().abs().max()) < 8
                    value, size = R.linear(attended[r].reshape(B, -1), values[r]["out"])
                    close(parts[r], value, size, "output projection")
                else:
                    (value, size), choice, _ = R.experts(seen[0][-1], layer.router.cpu(), values[r]["up"], values[r]["down"], top_k, 1.0)
                    assert torch.equal(layer.choice.cpu().long(), choice)
                    close(parts[r], value, size, "experts", 2.0 ** -15)
    with pytest.raises(ValueError, match="room for 3"):
        layer.step(x, stream)


def test_a_captured_layer():
    """A step in a graph, replayed with other inputs and eager work between."""
    announce("layer_step in a graph")
    E = _example()
    P, B, H = 2, 4, 256
    layer = E.Layer(P, B, H, 2, 1, 64, 64, 8, 2, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, stream = torch.zeros(B, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, H, dtype=torch.bfloat16, device="cuda")
    xs = [torch.randn(B, H, generator=g, device="cuda").bfloat16() for _ in range(4)]
    streams = [torch.randn(B, H, generator=g, device="cuda").bfloat16() for _ in range(4)]

    def run(i, call):
        layer.length.fill_(3)
        layer.used = 3
        x.copy_(xs[i])
        stream.copy_(streams[i])
        z = call()
        torch.cuda.synchronize()
        return z.clone(), stream.clone()

    want = [run(i, lambda: layer.step(x, stream)) for i in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, stream)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    layer.used = 3
    with torch.cuda.graph(graph):
        out = layer.step(x, stream)

    def replay():
        graph.replay()
        return out

    for i in (2, 0, 3, 1, 2):
        z, s = run(i, replay)
        assert torch.equal(z, want[i][0]) and torch.equal(s, want[i][1])
        eager = run((i + 1) % 4, lambda: layer.step(x, stream))
        assert torch.equal(eager[0], want[(i + 1) % 4][0])
