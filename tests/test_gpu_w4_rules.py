"""Products with 4-bit weights on both sides of every rule by which the calls choose a
kernel, and where offsets pass 32 bits.  Tolerances are those of test_gpu_w4.py and
test_gpu_w4_experts.py."""
from __future__ import annotations

import functools

import pytest
import torch

import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce
from test_gpu_w4 import close
from test_gpu_w4_experts import Layer

pytestmark = pytest.mark.gpu


@functools.lru_cache(maxsize=1)
def weights(K, N):
    packed, w = R.random_weights(N, K, torch.Generator().manual_seed(K + N), K ** -0.5)
    return packed.to(DEV), w


# one to four tiles of outputs to a workgroup, four of them with one workgroup to a
# compute unit (eight waves) and with more (four)
@pytest.mark.parametrize("K,N", [(2208, 900), (1184, 4790), (1184, 11190), (1184, 15990), (672, 32630)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 30, 45, 63, 130])
def test_linear(K, N, T):
    announce(f"w4_linear rules {T} {K} {N}")
    packed, w = weights(K, N)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(T)).bfloat16()
    out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ar.ar_w4_linear(x.to(DEV), packed, out[:-1])
    value, size = R.linear(x, w)
    close(out[:-1], value, size, "out")
    assert bool((out[-1] == 7.0).all())


# tokens, hidden, inner, experts, top_k: one and two tiles to a wave of the second
# product, with one and two groups of tokens; inner sizes past a block of chunks
@pytest.mark.parametrize("T,H,I,E,k", [
    (8, 1056, 32, 128, 16), (10, 1056, 32, 128, 16), (8, 4128, 32, 128, 16), (10, 4128, 32, 128, 16), (2, 64, 2208, 3, 2), (12, 64, 2208, 3, 2),
    (30, 96, 1120, 2, 2), (1, 96, 2208, 4, 3), (66, 64, 1056, 3, 2), (3, 2208, 64, 4, 2), (64, 1056, 64, 64, 8), (64, 2080, 32, 64, 8),
    (9, 64, 2208, 4, 1), (8, 544, 1056, 13, 8), (8, 160, 2208, 8, 8), (1, 96, 2208, 8, 8), (2, 1056, 64, 40, 3), (3, 2048, 32, 16, 4), (3, 2080, 32, 16, 4),
    (7, 32, 32, 15, 5), (5, 8192, 32, 3, 2), (6, 4128, 160, 5, 2), (1, 4128, 96, 4, 4), (8, 4096, 64, 6, 2),
    (9, 160, 1504, 20, 3), (9, 64, 2208, 8, 2), (30, 96, 2208, 2, 2), (64, 2080, 160, 64, 8), (64, 96, 64, 65, 8), (20, 160, 96, 3, 2), (64, 96, 288, 9, 5),
    (129, 64, 160, 7, 3), (24, 160, 544, 64, 8), (64, 96, 1056, 40, 6), (64, 1024, 608, 33, 4)])
def test_experts(T, H, I, E, k):
    announce(f"w4_experts rules {T} {H} {I} {E} {k}")
    layer = Layer(T, H, I, E, T + H + I)
    out, choice, weight = layer.run(k)
    (value, size), c, w = R.experts(layer.x, layer.router, layer.up, layer.down, k, 1.0)
    assert torch.equal(choice.long(), c) and bool(((weight.double() - w).abs() <= 2.0 ** -20 * w).all())
    close(out, value, size, "out", 2.0 ** -15)


@pytest.mark.parametrize("T,K", [(1, 76640), (1, 76960), (2, 38240), (2, 38560), (4, 19040), (4, 19360), (1, 32), (4, 160), (3, 2016), (4, 2080)])
def test_linear_of_long_rows(T, K):
    """Inputs that just fit into LDS, and some that do not; odd counts of chunks.  Of 602
    chunks a wave adds up to 301 instructions one after another: with an instruction's
    own terms and the waves' sums 350 times 2^-24, below 2^-15."""
    announce(f"w4_linear long rows {T} {K}")
    g = torch.Generator().manual_seed(K)
    packed, w = R.random_weights(37, K, g, K ** -0.5)
    x = torch.full((T, K + 40), float("inf"), dtype=torch.bfloat16)
    x[:, 5:5 + K] = torch.randn(T, K, generator=g).bfloat16()
    out = torch.empty(T, 37, dtype=torch.bfloat16, device=DEV)
    ar.ar_w4_linear(x.to(DEV)[:, 5:5 + K], packed.to(DEV), out)
    value, size = R.linear(x[:, 5:5 + K], w)
    close(out, value, size, "out", 2.0 ** -15 if K > 30000 else 2.0 ** -17)


def random_packed(tiles, n_in, g):
    """Packed weights made on the GPU: any codes, scales of 2^-4 to 1."""
    c = -(-n_in // 128)
    size = R.tile_bytes(n_in)
    packed = torch.randint(0, 256, (tiles, size), generator=g, dtype=torch.uint8, device=DEV)
    packed[:, 1024 * c:].remainder_(5).add_(123)
    if n_in % 128:
        packed[:, 1024 * (c - 1):1024 * c].view(tiles, 4, 256)[:, n_in % 128 // 32:] = 0
    return packed


@pytest.mark.parametrize("T", [2, 12, 40])
def test_linear_past_4_gib(T):
    announce(f"w4_linear past 4 GiB {T}")
    K, N = 28640, 300011
    tiles = -(-N // 16)
    g = torch.Generator(device=DEV).manual_seed(T)
    packed = random_packed(tiles, K, g)
    assert packed.numel() > 1 << 32
    far = (1 << 30) + 77  # elements from a token to the next
    base = torch.empty(far * (T - 1) + N, dtype=torch.bfloat16, device=DEV) if T == 2 else None
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    out = torch.empty(T, N, dtype=torch.bfloat16, device=DEV) if base is None else base.as_strided((T, N), (far, 1))
    ar.ar_w4_linear(x, packed, out)
    for tile in (0, 1, tiles // 2, tiles * 15 // 16, tiles - 2, tiles - 1):
        n = min(16, N - 16 * tile)
        value, size = R.linear(x.cpu(), R.values(packed[tile:tile + 1].cpu().numpy(), n, K))
        close(out[:, 16 * tile:16 * tile + n], value, size, f"tile {tile}")


@pytest.mark.parametrize("T", [1, 3, 20])
def test_experts_past_4_gib(T):
    announce(f"w4_experts past 4 GiB {T}")
    H, I, E, k = 2080, 4128, 512, 2
    g = torch.Generator(device=DEV).manual_seed(T)
    up, down = random_packed(E * I // 8, H, g).view(E, I // 8, -1), random_packed(E * H // 16, I, g).view(E, H // 16, -1)
    assert up.numel() > 1 << 32
    x = (0.02 * torch.randn(T, H, generator=g, device=DEV)).bfloat16()
    router = torch.randn(E, H, generator=g, device=DEV).bfloat16()
    router[511], router[509] = 8 * x[0], 7 * x[0]  # the last ones are taken
    out, choice = torch.empty(T, H, dtype=torch.bfloat16, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    router[:400] = 0
    weight = torch.empty(T, k, device=DEV)
    ws = torch.empty(ar.ar_w4_experts_workspace(T, H, I, E, k), dtype=torch.uint8, device=DEV)
    ar.ar_w4_experts(x, router, up, down, out, choice, weight, ws)
    logits = (x.cpu().double() @ router.cpu().double().T).float()
    c = R.choose(logits, k)
    assert torch.equal(choice.cpu().long(), c)
    taken = c.unique().tolist()
    assert max(taken) > 500
    index = {e: i for i, e in enumerate(taken)}
    (value, size), local, w = R.experts(x.cpu(), router[taken].cpu(), [R.values(up[e].cpu().numpy(), 2 * I, H) for e in taken],
                                        [R.values(down[e].cpu().numpy(), H, I) for e in taken], k, 1.0)
    if len(taken) >= k:
        assert torch.equal(local, c.apply_(lambda e: index[e]))
    close(out, value, size, "out", 2.0 ** -15)


@pytest.mark.parametrize("T,H,I", [(3, 64, 160), (8, 64, 160), (8, 1056, 160), (9, 64, 160), (9, 1056, 160), (40, 64, 416), (8, 64, 800)])
def test_an_expert_of_nan(T, H, I):
    """Weights of NaN in either product reach the tokens that take the expert, and no other."""
    announce(f"w4_experts with an expert of NaN {T} {H} {I}")
    E, k = 40, 3
    layer = Layer(T, H, I, E, T + H)
    clean, c, _ = layer.run(k)
    for packed, scales in ((layer.packed_up, 256 * -(-H // 512)), (layer.packed_down, 256 * -(-I // 512))):
        kept, bad = packed.clone(), int(c[0, 1])
        packed[bad, :, -scales:] = 255
        out, choice, _ = layer.run(k)
        takes = (choice == bad).any(1)
        assert torch.equal(choice, c) and 0 < int(takes.sum()) < T
        assert bool(torch.isnan(out.cpu()[takes]).all()) and torch.equal(out.cpu()[~takes], clean.cpu()[~takes])
        packed.copy_(kept)


@pytest.mark.parametrize("T", [1, 6, 20])
def test_equal_logits_of_a_large_router(T):
    announce(f"w4_experts with equal logits {T}")
    layer = Layer(T, 544, 32, 70, 5)
    layer.router[:] = layer.router[3]
    layer.router[40] *= 2
    layer.router[50] = -layer.router[40]
    _, choice, weight = layer.run(5)
    for t in range(T):
        assert choice[t, 0].item() in (40, 50) and choice[t, 1:].tolist() == [0, 1, 2, 3]
        assert weight[t, 1:].unique().numel() == 1


def test_kernels_with_much_lds_in_a_graph():
    """Inputs of 150 KB held in LDS, and sums of 64 tokens there, captured and replayed."""
    announce("w4 graphs with much LDS")
    g = torch.Generator(device=DEV).manual_seed(9)
    n = lambda *s, size=1.0: (size * torch.randn(*s, generator=g, device=DEV)).bfloat16()  # noqa: E731
    T, H, I, E, k = 64, 96, 96, 9, 5
    K, N = 76640, 37
    wide, up, down = random_packed(3, K, g), random_packed(E * I // 8, H, g).view(E, I // 8, -1), random_packed(E * H // 16, I, g).view(E, H // 16, -1)
    x, y, tokens, out = n(1, K), n(1, N), n(T, H), n(T, H)
    router, choice, weight = n(E, H), torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    ws = torch.empty(ar.ar_w4_experts_workspace(T, H, I, E, k), dtype=torch.uint8, device=DEV)

    def run():
        ar.ar_w4_linear(x, wide, y)
        ar.ar_w4_experts(tokens, router, up, down, out, choice, weight, ws)

    inputs = [(n(1, K), n(T, H)) for _ in range(3)]
    want = []
    for a, b in inputs:
        x.copy_(a)
        tokens.copy_(b)
        run()
        want.append((y.clone(), out.clone(), choice.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in (1, 0, 2, 1):
        x.copy_(inputs[i][0])
        tokens.copy_(inputs[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i][0]) and torch.equal(out, want[i][1]) and torch.equal(choice, want[i][2])
        run()
        assert torch.equal(y, want[i][0]) and torch.equal(out, want[i][1])
