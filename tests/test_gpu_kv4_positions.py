"""Sequences longer than their rows of the page table: a query's position comes
from the length as it is given, and only the tokens past the table's last entry
are unseen."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import announce
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,heads,hk,m,n,entries,window", [
    (64, 4, 2, 5, 100, 2, 0), (64, 4, 2, 5, 67, 2, 0), (128, 8, 2, 3, 100, 2, 50), (128, 8, 2, 40, 100, 2, 20), (256, 4, 1, 6, 69, 2, 9),
    (128, 8, 1, 2, 6000, 150, 0), (128, 8, 1, 4, 6000, 150, 1300), (64, 4, 2, 30, 300, 2, 40),
    (64, 48, 16, 1100, 1200, 11, 0), (128, 32, 8, 1100, 1300, 11, 90), (256, 16, 8, 1100, 1133, 11, 300)])
def test_more_tokens_than_entries(D, heads, hk, m, n, entries, window):
    announce(f"kv4 positions {D} {heads} {hk} {m} {n} {entries} {window}")
    page = 32 if n < 1000 else 64
    c = Case([m, m - 1], [n, n - 3], heads, hk, D, page, window)
    c.table[:, entries:] = 1 << 30  # no page: the same tokens unseen, positions as given
    whole = c.table
    c.check(*c.run())
    c.table = whole[:, :entries].contiguous()
    got = c.run()
    c.table = whole
    c.check(*got)


@pytest.mark.parametrize("D,heads,hk,m", [(64, 4, 2, 3), (128, 8, 2, 1), (256, 4, 1, 2), (128, 32, 8, 1100)])
def test_the_longest_length(D, heads, hk, m):
    """Positions up to 2^31 - 2, over a table of 96 tokens."""
    announce(f"kv4 longest {D} {heads} {hk} {m}")
    c = Case([m, m, m], [96, 96, 96], heads, hk, D, 32)
    longest = 2 ** 31 - 1
    c.kvlens = [longest, longest, 96 + m]  # the last: every query sees all 96
    out, lse = c.run(max_kv=96)
    lost = torch.full((3, -(-m // 32)), 1 << 30, dtype=torch.int32)
    c.table, c.kvlens = torch.cat([c.table, lost], 1), [96 + m] * 3  # every query sees all 96
    c.check(out, lse)


@pytest.mark.parametrize("window", [1, 1000, 2 ** 31 - 1 - 200, 2 ** 31 - 1 - 50])
def test_the_longest_length_with_a_window(window):
    D, page = 64, 32
    c = Case([2], [96], 2, 1, D, page)
    n = 2 ** 31 - 1
    c.kvlens, c.window = [n], window
    out, lse = c.run(max_kv=96)
    for i in range(2):
        first = max(0, n - 2 + i - window + 1)  # the first token that query i sees
        if first >= 96:
            assert not out[i].any() and bool((lse[i] == -math.inf).all())
            continue
        one = Case([2], [96], 2, 1, D, page)
        one.qlens, one.kvlens, one.start, one.T = [1], [96], torch.tensor([i, i + 1], dtype=torch.int32), 2
        one.window = 96 - first
        one.check(out, lse)
