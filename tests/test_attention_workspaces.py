"""CPU tests of the attention operators' workspace sizes: they never fall as a
call grows, so that the workspace of a program's largest call serves all."""
from __future__ import annotations

import random

import pytest

from allreduce_reduction_way_amd import ar


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (64, 8, 128), (28, 4, 64), (1, 1, 256), (12, 12, 64), (96, 8, 256)])
def test_attention_workspace_never_falls(heads, kv_heads, dim):
    rng = random.Random(heads * dim)
    batches = sorted({1, 2, 63, 64, 65, 127, 128, 511, 512, 513, 1024} | {rng.randint(1, 2000) for _ in range(12)})
    queries = sorted({0, 1, 2, 5, 6, 17, 64, 65, 500, 2048} | {rng.randint(1, 3000) for _ in range(4)})
    tokens = sorted({0, 1, 255, 256, 511, 512, 513, 4095, 8192, 200003, 2 ** 31 - 1} | {rng.randint(1, 1 << 18) for _ in range(6)})

    def size(b, q, kv):
        return ar.ar_kv4_attention_workspace(b, b * q, q, kv, heads, kv_heads, dim)

    for axes in ((batches, queries, tokens), (queries, tokens, batches), (tokens, batches, queries)):
        for y in axes[1]:
            for z in axes[2]:
                last = 0
                for x in axes[0]:
                    sizes = {id(axes[0]): x, id(axes[1]): y, id(axes[2]): z}
                    n = size(sizes[id(batches)], sizes[id(queries)], sizes[id(tokens)])
                    assert n >= max(16, last), (x, y, z)
                    last = n


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_gradient_workspace_never_falls(dim):
    tokens = [0, 1, 2, 3, 7, 100, 511, 512, 513, 1023, 1024, 1025, 1366, 2047, 2048, 2049, 4095, 4096, 4097, 100000]
    heads = [0, 1, 2, 7, 8, 9, 16, 40, 64, 100]

    def size(t, hq, hk):
        return ar.ar_qk_norm_rope_bwd_workspace(t, hq, hk, dim)

    for a in heads:
        for b in heads:
            for lo, hi in zip(tokens, tokens[1:]):
                assert 8 * dim <= size(lo, a, b) <= size(hi, a, b), (lo, hi, a, b)
    for t in tokens:
        for a in heads:
            for lo, hi in zip(heads, heads[1:]):
                assert size(t, a, lo) <= size(t, a, hi) and size(t, lo, a) <= size(t, hi, a), (t, a, lo, hi)
