"""One decode step of an attention layer on P tensor-parallel ranks, emulated on
one GPU as the library's own calls emulate them.

Each rank has its share of the heads: it norms and turns its queries and keys
(ar_qk_norm_rope), quantises the new token's keys and values into its 4-bit
cache (ar_kv4_write), attends over the cache (ar_kv4_attention), and multiplies
the result with its rows of the output projection.  The ranks' partial sums are
added up by the write-mode all-reduce (ar_oneshot_write_bcast).

    python examples/decode_share.py [--ranks 8] [--batch 8] [--tokens 1000]
"""
from __future__ import annotations

import argparse
import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
from allreduce_reduction_way_amd import ar  # noqa: E402

PAGE = 64


class Layer:
    """Weights, caches and buffers of one layer, for all ranks."""

    def __init__(self, ranks: int, batch: int, heads: int, kv_heads: int, dim: int, tokens: int, seed: int = 0):
        """`heads` and `kv_heads` of each rank; room for `tokens` tokens of each
        of `batch` sequences."""
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, size=1.0):
            return (size * torch.randn(*shape, generator=g, device="cuda")).bfloat16()

        self.P, self.B, self.hq, self.hk, self.D = ranks, batch, heads, kv_heads, dim
        self.hidden = ranks * heads * dim
        self.q_weight, self.k_weight = 1 + normal(dim, size=0.1), 1 + normal(dim, size=0.1)
        self.projection = [normal(heads * dim, self.hidden, size=self.hidden ** -0.5) for _ in range(ranks)]
        angle = torch.arange(tokens, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        per = -(-tokens // PAGE)  # pages of a sequence
        self.max_kv = per * PAGE
        self.room, self.used = tokens, 0  # tokens of a sequence: that fit, that are cached
        order = torch.randperm(batch * per, generator=g, device="cuda")
        self.table = order.reshape(batch, per).int()
        self.cache = [torch.zeros(batch * per, kv_heads, PAGE // 32, 34 * dim, dtype=torch.uint8, device="cuda")
                      for _ in range(ranks)]
        self.length = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.q_start = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
        self.out = torch.empty(batch, heads, dim, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(batch, heads, device="cuda")
        nbytes = ar.ar_kv4_attention_workspace(batch, batch, 1, self.max_kv, heads, kv_heads, dim)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.sums = [torch.empty(batch, self.hidden, dtype=torch.bfloat16, device="cuda") for _ in range(ranks)]

    def fill(self, keys, values) -> None:
        """Caches a prompt: keys and values (tokens, kv_heads, dim) of each rank
        and sequence, keys normed and turned already."""
        self._take(keys[0][0].shape[0] - self.used)
        for r in range(self.P):
            for b in range(self.B):
                k, v = keys[r][b], values[r][b]
                at = torch.arange(k.shape[0], device="cuda")
                slots = self.table[b].long()[at // PAGE] * PAGE + at % PAGE
                ar.ar_kv4_write(k, v, slots, self.cache[r], PAGE)
        self.length.fill_(self.used)

    def _take(self, tokens: int) -> None:
        """Room for so many more tokens of each sequence: pages past the table's
        would be looked up otherwise."""
        if self.used + tokens > self.room:
            raise ValueError(f"{self.used + tokens} tokens, there is room for {self.room}")
        self.used += tokens

    def step(self, qkv) -> list:
        """One new token of every sequence: qkv[r] (batch, heads + 2 kv_heads,
        dim) is what rank r's projection gave, normed and turned in place.
        Returns every rank's copy of the summed output (batch, hidden)."""
        hq, hk = self.hq, self.hk
        self._take(1)
        positions = self.length.long()
        slots = self.table.long().gather(1, (positions // PAGE)[:, None])[:, 0] * PAGE + positions % PAGE
        self.length += 1
        partial = []
        for r in range(self.P):
            q, k, v = qkv[r][:, :hq], qkv[r][:, hq:hq + hk], qkv[r][:, hq + hk:]
            ar.ar_qk_norm_rope(q, k, self.q_weight, self.k_weight, self.cos_sin, positions)
            ar.ar_kv4_write(k, v, slots, self.cache[r], PAGE)
            ar.ar_kv4_attention(q, self.cache[r], self.table, self.q_start, self.length, self.out, self.lse,
                                self.workspace, page_size=PAGE, kv_heads=hk, max_q=1, max_kv=self.max_kv)
            partial.append(self.out.reshape(self.B, -1) @ self.projection[r])
        ar.ar_oneshot_write_bcast(partial, self.sums)
        return self.sums


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--tokens", type=int, default=1000)
    a = p.parse_args()
    heads, kv_heads, dim, steps = 8, 1, 128, 16
    layer = Layer(a.ranks, a.batch, heads, kv_heads, dim, a.tokens + steps)

    def normal(*shape):
        return torch.randn(*shape, device="cuda").bfloat16()

    layer.fill([[normal(a.tokens, kv_heads, dim) for _ in range(a.batch)] for _ in range(a.ranks)],
               [[normal(a.tokens, kv_heads, dim) for _ in range(a.batch)] for _ in range(a.ranks)])
    for n in range(steps):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        qkv = [normal(a.batch, heads + 2 * kv_heads, dim) for _ in range(a.ranks)]
        start.record()
        out = layer.step(qkv)
        end.record()
        end.synchronize()
    print(f"{a.ranks} ranks, {a.batch} sequences of {a.tokens + steps} tokens: the last of {steps} steps took "
          f"{1000 * start.elapsed_time(end):.0f} us; output {tuple(out[0].shape)}, rms {out[0].float().square().mean().sqrt():.3f}")


if __name__ == "__main__":
    main()
