"""What the 4-bit cache holds where no query looks changes no bit of the
attention's results: pages that are used in part hold whatever memory held
before.  Every scale byte occurs there, among them 253 and 254 (2^126 and 2^127,
whose codes go beyond bf16) and 255 (NaN)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from gpu_util import announce
from test_gpu_kv4_attention import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # qlens, kvlens, heads, kv_heads, D, page, window
    ([1, 1], [70, 33], 4, 2, 64, 64, 0),
    ([1, 4], [300, 130], 8, 2, 128, 128, 0),
    ([3, 1], [45, 200], 4, 1, 256, 64, 0),
    ([2, 3], [500, 333], 8, 2, 128, 64, 100),
    ([5, 2], [150, 90], 12, 2, 64, 32, 20),
    ([1], [5003], 8, 1, 128, 256, 0),                  # split over workgroups
    ([1100, 1090, 2], [1203, 1187, 1], 48, 16, 64, 64, 0),   # every wave has rows of its own
    ([1100, 1090, 2], [1103, 1187, 1], 32, 8, 128, 64, 0),
    ([1100, 1090, 2], [1133, 1120, 1], 16, 8, 256, 64, 40)]


def _unseen(c):
    """(pages, 1, tiles, 32): places that no query of any sequence sees."""
    seen = np.zeros((c.pages, c.page), dtype=bool)
    for b, (m, n) in enumerate(zip(c.qlens, c.kvlens)):
        first = max(0, n - m - c.window + 1) if c.window else 0
        j = np.arange(first, n)
        seen[c.table[b].numpy()[j // c.page], j % c.page] = True
    return ~seen.reshape(c.pages, 1, -1, 32)


@pytest.mark.parametrize("shape", SHAPES)
def test_unseen_bytes_change_nothing(shape):
    announce(f"kv4 unseen {shape}")
    c = Case(*shape)
    away = _unseen(c)
    for codes, scales in ((c.kc, c.kb), (c.vc, c.vb)):
        codes[np.broadcast_to(away, codes.shape[:-1])] = 0
        scales[np.broadcast_to(away, scales.shape[:-1])] = 2
    want = c.run()
    rng = np.random.default_rng(1)
    for what in (253, 254, 255, "any"):
        for codes, scales in ((c.kc, c.kb), (c.vc, c.vb)):
            at = np.broadcast_to(away, codes.shape[:-1])
            n = int(at.sum())
            codes[at] = rng.integers(0, 16, (n, codes.shape[-1]))
            scales[at] = rng.integers(0, 256, (n, scales.shape[-1])) if what == "any" else what
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), what
    if sum(c.qlens) < 100:
        c.check(*want)


@pytest.mark.parametrize("D,heads,hk,m,n", [(64, 4, 2, 6, 70), (128, 8, 2, 5, 100), (256, 4, 1, 3, 45), (64, 48, 16, 1100, 1200),
                                            (128, 32, 8, 1100, 1100), (256, 16, 8, 1100, 1133)])
@pytest.mark.parametrize("byte", [253, 254])
def test_values_beyond_bf16_reach_only_who_sees_them(D, heads, hk, m, n, byte):
    announce(f"kv4 beyond bf16 {D} {heads} {hk} {m} {n} {byte}")
    c = Case([m, m], [n, n - 7], heads, hk, D, 64)
    t = n - 2  # the last two queries of the first sequence see it
    page, in_page = c.table[0, t // 64], t % 64
    c.vc[page, 0, in_page // 32, in_page % 32] = 7
    want = c.run()
    c.vb[page, 0, in_page // 32, in_page % 32, 1] = byte
    got = c.run()
    touched = torch.zeros(want[0].shape, dtype=torch.bool)
    touched[m - 2:m, :heads // hk, 32:64] = True
    assert torch.equal(got[0][~touched], want[0][~touched]) and torch.equal(got[1], want[1])
    assert not torch.isfinite(got[0][touched]).any()
