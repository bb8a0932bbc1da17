"""The precision of the 4-bit cache's scores, seen in lse, which has no rounding of
weights in it.

A key's codes times their scale and a query are bf16 as they are, so that products
are exact in binary32 (8 and 2 significant bits); what is off is their sum.

Sums that binary32 holds.  Queries and keys of few bits make every partial sum, in
whatever order, exact.  Then each score is exact, and lse is off by: scale log2(e) (a
rounded product, 2^-24 each, and a rounded factor), the maximum added to the log2 of the
sum, ln 2 and the product with it: six roundings of 2^-24 of lse at most, and for the sum
of weights, relative: one rounding for every token that a lane adds (a quarter
of them at most), 2^-24 each, and 40 for exponentials and joins.

Any queries.  Each of the D - 1 additions is off by at most 2^-23 (either
neighbour) of the sum of the terms' sizes: ds = D 2^-23 scale max_j sum_c |q_c k_jc|,
over the tokens that a row sees."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_util import announce
from test_gpu_kv4_attention import SHAPES, Case

pytestmark = pytest.mark.gpu


def _lse(c, scale):
    """lse in 64 bits (tokens, heads), and ds of every row."""
    lse, ds = torch.zeros(c.T, c.heads, dtype=torch.float64), torch.zeros(c.T, c.heads, dtype=torch.float64)
    k, q = R.values(c.kc, c.kb), c.q().double()
    for b, (m, n) in enumerate(zip(c.qlens, c.kvlens)):
        s0, j = int(c.start[b]), np.arange(n)
        page = c.table[b].numpy()[j // c.page]
        pos = n - m + torch.arange(m)
        seen = torch.arange(n) <= pos[:, None]
        if c.window:
            seen &= torch.arange(n) > pos[:, None] - c.window
        for h in range(c.heads):
            kk = torch.from_numpy(k[page, h // (c.heads // c.hk), j % c.page // 32, j % 32]).reshape(n, c.D)
            x = (scale * q[s0:s0 + m, h] @ kk.T).masked_fill(~seen, -float("inf"))
            lse[s0:s0 + m, h] = torch.logsumexp(x, 1) if n else -float("inf")
            if n:
                ds[s0:s0 + m, h] = (scale * q[s0:s0 + m, h].abs() @ kk.abs().T).masked_fill(~seen, 0).amax(1) * c.D * 2.0 ** -23
    return lse, ds


def _close(c, got, want, ds):
    none = torch.isinf(want)
    assert torch.equal(torch.isinf(got), none)
    off = torch.where(none, 0.0, (got.double() - want).abs())
    tol = ds + 2.0 ** -24 * (6 * (1 + torch.where(none, 0.0, want).abs()) + max(c.kvlens) / 4 + 40)
    assert bool((off <= tol).all()), float((off / tol).max())


PROMPTS = [([1100, 1090, 2], [1203, 1187, 1], 48, 16, 64, 64, 0), ([1100, 1090, 2], [1103, 1187, 1], 32, 8, 128, 64, 0),
           ([1100, 1090, 2], [1133, 1120, 1], 16, 8, 256, 64, 40)]


@pytest.mark.parametrize("shape", SHAPES + PROMPTS)
def test_sums_that_binary32_holds(shape):
    """A channel of 2^15 among others below 2^7: partial sums stay below 2^20 halves."""
    announce(f"exact scores {shape}")
    c = Case(*shape)
    c.kb[:] = 127
    rng = np.random.default_rng(7)
    q = rng.integers(-127, 128, (c.T, c.heads, c.D)).astype(np.float64)
    big = rng.integers(0, c.D, (c.T, c.heads))
    q[np.arange(c.T)[:, None], np.arange(c.heads), big] = rng.choice([-1.25, -1.0, 1.0, 1.25], big.shape) * 2.0 ** 15
    c.flat[:, :c.heads * c.D] = torch.from_numpy(q.reshape(c.T, -1)).bfloat16()
    assert torch.equal(c.q().double(), torch.from_numpy(q))
    scale = 2.0 ** -12
    want, _ = _lse(c, scale)
    _close(c, c.run(scale=scale)[1], want, 0.0)


@pytest.mark.parametrize("shape", SHAPES + PROMPTS)
def test_any_queries(shape):
    announce(f"scores {shape}")
    c = Case(*shape)
    want, ds = _lse(c, c.D ** -0.5)
    _close(c, c.run()[1], want, ds)
