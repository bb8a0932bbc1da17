"""One decode step of a whole layer on P tensor-parallel ranks, emulated on one GPU
as the library's own calls emulate them: attention, then a mixture of experts.

The residual stream is on every rank.  Each rank's products have weights of 4 bits:
its queries, keys and values (ar_w4_linear), its heads' norms and rotation
(ar_qk_norm_rope), its 4-bit cache (ar_kv4_write) and attention over it
(ar_kv4_attention), its rows of the output projection (ar_w4_linear), and its share
of every expert (ar_w4_experts).  After both halves the ranks' partial outputs are
added up, normed and added to the stream, and the next half's input is normed, in one
pass (ar_block_norm).

    python examples/layer_step.py [--ranks 8] [--batch 8] [--tokens 1000]
"""
from __future__ import annotations

import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
from allreduce_reduction_way_amd import ar  # noqa: E402

PAGE = 64


def pack(w):
    """Weights (..., n_out, n_in) in 4 bits."""
    *lead, n_out, n_in = w.shape
    packed = torch.empty(*lead, -(-n_out // 16), ar.ar_w4_bytes(16, n_in), dtype=torch.uint8, device=w.device)
    for one, to in zip(w.reshape(-1, n_out, n_in), packed.reshape(-1, *packed.shape[-2:])):
        ar.ar_w4_pack(one, to)
    return packed


class Rank:
    """One rank's weights, cache and buffers."""

    def __init__(self, normal, batch, hidden, heads, kv_heads, dim, inner, experts, pages):
        self.qkv_weight = pack(normal((heads + 2 * kv_heads) * dim, hidden, size=hidden ** -0.5))
        self.out_weight = pack(normal(hidden, heads * dim, size=(heads * dim) ** -0.5))
        self.gate_up = pack(normal(experts, 2 * inner, hidden, size=hidden ** -0.5))
        self.down = pack(normal(experts, hidden, inner, size=inner ** -0.5))
        self.cache = torch.zeros(pages, kv_heads, PAGE // 32, 34 * dim, dtype=torch.uint8, device="cuda")
        empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.qkv = empty(batch, heads + 2 * kv_heads, dim)
        self.attended = empty(batch, heads, dim)
        self.partial = empty(batch, hidden)


class Layer:
    """Weights, caches and buffers of one layer, for all ranks."""

    def __init__(self, ranks: int, batch: int, hidden: int, heads: int, kv_heads: int, dim: int, inner: int, experts: int, top_k: int,
                 tokens: int, seed: int = 0):
        """`heads`, `kv_heads` and `inner` of each rank; room for `tokens` tokens
        of each of `batch` sequences."""
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, size=1.0):
            return (size * torch.randn(*shape, generator=g, device="cuda")).bfloat16()

        self.P, self.B, self.hidden, self.hq, self.hk, self.D, self.top_k = ranks, batch, hidden, heads, kv_heads, dim, top_k
        per = -(-tokens // PAGE)
        self.room, self.used, self.max_kv = tokens, 0, per * PAGE
        self.table = torch.randperm(batch * per, generator=g, device="cuda").reshape(batch, per).int()
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.q_start = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        angle = torch.arange(tokens, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.q_weight, self.k_weight = 1 + normal(dim, size=0.1), 1 + normal(dim, size=0.1)
        # norms after each half and before the other one, and the halves' gates
        self.post = [1 + normal(hidden, size=0.1) for _ in range(2)]
        self.pre = [1 + normal(hidden, size=0.1) for _ in range(2)]
        self.gate = [(0.5 + normal(hidden, size=0.1)) for _ in range(2)]
        self.router = normal(experts, hidden, size=hidden ** -0.5)
        self.ranks = [Rank(normal, batch, hidden, heads, kv_heads, dim, inner, experts, batch * per) for _ in range(ranks)]
        self.choice = torch.empty(batch, top_k, dtype=torch.int32, device="cuda")
        self.weight = torch.empty(batch, top_k, device="cuda")
        self.lse = torch.empty(batch, heads, device="cuda")
        self.inputs = [torch.empty(batch, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(2)]  # of the experts, of the next layer
        size = max(ar.ar_kv4_attention_workspace(batch, batch, 1, self.max_kv, heads, kv_heads, dim),
                   ar.ar_w4_experts_workspace(batch, hidden, inner, experts, top_k))
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")

    def join(self, half: int, stream) -> torch.Tensor:
        """The ranks' partial outputs of a half into the stream (in place), and the norm before what comes next."""
        z = self.inputs[half]
        ar.ar_block_norm([r.partial for r in self.ranks], stream, stream, z, post_weight=self.post[half], gate=self.gate[half],
                         pre_weight=self.pre[1 - half])
        return z

    def step(self, x, stream) -> torch.Tensor:
        """One new token of every sequence: x (batch, hidden) is the normed input, `stream` the residual stream, which is
        updated.  Returns the next layer's normed input.  Captured and replayed, when the room is not looked at any
        more, a step past it writes to no cache and gives NaN."""
        if self.used + 1 > self.room:
            raise ValueError(f"{self.used + 1} tokens, there is room for {self.room}")
        self.used += 1
        positions = self.length.long()
        pages = self.table.long().gather(1, (positions // PAGE).clamp(max=self.table.shape[1] - 1)[:, None])[:, 0]
        slots = torch.where(positions < self.room, pages * PAGE + positions % PAGE, -1)
        self.length += 1
        for r in self.ranks:
            ar.ar_w4_linear(x, r.qkv_weight, r.qkv.view(self.B, -1))
            q, k, v = r.qkv[:, :self.hq], r.qkv[:, self.hq:self.hq + self.hk], r.qkv[:, self.hq + self.hk:]
            ar.ar_qk_norm_rope(q, k, self.q_weight, self.k_weight, self.cos_sin, positions)
            ar.ar_kv4_write(k, v, slots, r.cache, PAGE)
            ar.ar_kv4_attention(q, r.cache, self.table, self.q_start, self.length, r.attended, self.lse, self.workspace, page_size=PAGE,
                                kv_heads=self.hk, max_q=1, max_kv=self.max_kv)
            ar.ar_w4_linear(r.attended.view(self.B, -1), r.out_weight, r.partial)
        z = self.join(0, stream)
        for r in self.ranks:
            ar.ar_w4_experts(z, self.router, r.gate_up, r.down, r.partial, self.choice, self.weight, self.workspace)
        return self.join(1, stream)


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--tokens", type=int, default=1000)
    a = p.parse_args()
    hidden, experts, top_k, steps = 5120, 64, 6, 16
    layer = Layer(a.ranks, a.batch, hidden, 8, 1, 128, 192, experts, top_k, a.tokens + steps)
    layer.length.fill_(a.tokens)  # of keys and values that are zeros
    layer.used = a.tokens
    stream = torch.randn(a.batch, hidden, device="cuda").bfloat16()
    x = torch.randn(a.batch, hidden, device="cuda").bfloat16()
    for _ in range(steps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        x = layer.step(x, stream)
        end.record()
        end.synchronize()
    print(f"{a.ranks} ranks, {a.batch} sequences of {a.tokens + steps} tokens: the last of {steps} steps took "
          f"{1000 * start.elapsed_time(end):.0f} us; stream {tuple(stream.shape)}, rms {stream.float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
