"""Scores so large that one's own rounding is many powers of two: the softmax is
the mean of the values at the largest score, and lse is that score.

Queries have one channel that is not zero, so that a score is one product, exact
in binary32, and every pair of scores is equal or apart by more than any weight
can bridge (2^20 at least).  Equal weights are rounded equally, so the output is off by
its own rounding (2^-8) and binary32 sums (2^-15 of sum |v|); lse by a few
binary32 roundings, 2^-20 of it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_util import announce
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [
    ([1, 3], [70, 200], 4, 2, 64, 64, 0),
    ([1, 2], [300, 131], 8, 2, 128, 64, 0),
    ([2, 2], [45, 100], 4, 1, 256, 32, 30),
    ([1], [5003], 8, 1, 128, 256, 0),                        # joined from ranges
    ([1100, 1090, 2], [1200, 1187, 1], 48, 16, 64, 64, 0),   # every wave has rows of its own
    ([1100, 1090, 2], [1103, 1187, 1], 32, 8, 128, 64, 0),
    ([1100, 1090, 2], [1133, 1120, 1], 16, 8, 256, 64, 0)])
def test_scores_beyond_the_exponential(shape):
    qlens, kvlens, heads, hk, D, page, window = shape
    announce(f"kv4 large scores {shape}")
    c = Case(*shape)
    c.kb[:] = 127
    c.kc[..., 1] = np.random.default_rng(3).permutation(c.kc[..., 0].ravel()).reshape(c.kc[..., 0].shape)
    size = 2.0 ** np.array([26, 30, 31, 32, 33, 36, 50, 90, 120])
    rng = np.random.default_rng(5)
    q = np.zeros((c.T, heads, D))
    # sign, channel and size by row
    q[np.arange(c.T)[:, None], np.arange(heads), rng.integers(0, 2, (c.T, heads))] = \
        rng.choice(size, (c.T, heads)) * rng.choice([-1.0, 1.0], (c.T, heads)) * rng.choice([1.0, 1.25, 1.9921875], (c.T, heads))
    c.flat[:, :heads * D] = torch.from_numpy(q.reshape(c.T, -1)).bfloat16()
    out, lse = c.run(scale=0.75)
    k, v = R.values(c.kc, c.kb), R.values(c.vc, c.vb)
    query = c.q().double()
    for b, (m, n) in enumerate(zip(qlens, kvlens)):
        s0, j = int(c.start[b]), np.arange(n)
        pages = c.table[b].numpy()[j // page]
        pos = n - m + torch.arange(m)
        seen = torch.arange(n) <= pos[:, None]
        if window:
            seen &= torch.arange(n) > pos[:, None] - window
        some = seen.any(1)
        for h in range(heads):
            at = (pages, h // (heads // hk), j % page // 32, j % 32)
            kk, vv = torch.from_numpy(k[at]), torch.from_numpy(v[at])
            s = (0.75 * query[s0:s0 + m, h, :2] @ kk[:, :2].T).masked_fill(~seen, -float("inf"))
            top = s.amax(1, keepdim=True)
            p = ((s == top) & seen).double()
            count = p.sum(1, keepdim=True)
            want, size_v = (p @ vv / count)[some], (p @ vv.abs() / count)[some]
            got = out[s0:s0 + m, h].double()[some]
            assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * size_v).all()), (b, h)
            wl = (top[:, 0] + torch.log(count[:, 0]))[some]
            gl = lse[s0:s0 + m, h].double()[some]
            assert bool(((gl - wl).abs() <= 2.0 ** -20 * (1 + wl.abs())).all()), (b, h)
