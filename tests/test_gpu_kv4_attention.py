"""GPU parity of attention over the 4-bit cache against the 64-bit definition.

Tolerances.  Scores: a query is held in two e4m3 parts, to 2^-21 of its largest
element, and products are added in binary32 (at most 256 terms, 2^-16 of their
sizes is more than any order of adding loses); with the largest query element
and the sum of a key's magnitudes as the size, ds = 2^-15 scale |q|_max |k|_1.
Weights are rounded to bf16: 2^-8 of each, with 2 ds (numerator and sum) and
2^-15 for the exponential and the sums.  The output adds 2^-8 of itself.  lse: ds
and 2^-18 of (1 + |lse|)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu


class Case:
    """Queries, a cache of random codes and scales, pages in any order."""

    def __init__(self, qlens, kvlens, heads, kv_heads, D, page, window=0, seed=0, odd=False, q_size=2.0):
        rng = np.random.default_rng(seed + 1000 * D + heads)
        g = torch.Generator().manual_seed(seed + D)
        self.qlens, self.kvlens, self.window, self.page = qlens, kvlens, window, page
        self.heads, self.hk, self.D = heads, kv_heads, D
        used = [-(-n // page) for n in kvlens]
        self.pages = sum(used) + 2
        shape = (self.pages, kv_heads, page // 32, 32)
        self.kc, self.vc = rng.integers(0, 16, (*shape, D)), rng.integers(0, 16, (*shape, D))
        self.kb, self.vb = rng.integers(122, 128, (*shape, D // 32)), rng.integers(122, 129, (*shape, D // 32))
        per = max(1, max(used))
        order = rng.permutation(self.pages)[:sum(used)]
        self.table = torch.full((len(kvlens), per), 1 << 30, dtype=torch.int32)  # unused entries: no page
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = torch.from_numpy(order[at:at + n].astype(np.int32))
            at += n
        self.T = sum(qlens)
        pad = 1 if odd else 0
        flat = torch.zeros(self.T, heads * D + pad, dtype=torch.bfloat16)
        flat[:, :heads * D] = (q_size * torch.randn(self.T, heads * D, generator=g)).bfloat16()
        self.flat = flat
        self.start = torch.tensor([0, *np.cumsum(qlens)], dtype=torch.int32)

    def q(self):
        return self.flat[:, :self.heads * self.D].unflatten(1, (self.heads, self.D))

    def run(self, ws=None, max_q=None, max_kv=None, scale=None, stream=None, odd_out=False):
        d = lambda x: x.to(DEV)  # noqa: E731
        mq, mk = max_q or max(self.qlens), max(self.kvlens) if max_kv is None else max_kv
        if ws is None:
            ws = torch.zeros(ar.ar_kv4_attention_workspace(len(self.qlens), self.T, mq, mk, self.heads, self.hk, self.D),
                             dtype=torch.uint8, device=DEV)
        cache = d(torch.from_numpy(R.pack(self.kc, self.kb, self.vc, self.vb)))
        pad = 1 if odd_out else 0
        store = torch.full((self.T, self.heads * self.D + pad), 7.0, dtype=torch.bfloat16, device=DEV)
        out = store[:, :self.heads * self.D].unflatten(1, (self.heads, self.D))
        lse = torch.full((self.T, self.heads), 7.0, device=DEV)
        q = d(self.flat)[:, :self.heads * self.D].unflatten(1, (self.heads, self.D))
        ar.ar_kv4_attention(q, cache, d(self.table), d(self.start), d(torch.tensor(self.kvlens, dtype=torch.int32)), out, lse,
                            ws, page_size=self.page, kv_heads=self.hk, max_q=mq, max_kv=mk, window=self.window, scale=scale,
                            stream=stream)
        torch.cuda.synchronize()
        if pad:
            assert bool((store[:, -1] == 7).all())
        return out.cpu(), lse.cpu()

    def check(self, out, lse, scale=None, unseen=()):
        """`unseen`: (sequence, token) pairs that no query sees."""
        scale = self.D ** -0.5 if scale is None else scale
        group, tpp = self.heads // self.hk, self.page // 32
        k, v = R.values(self.kc, self.kb), R.values(self.vc, self.vb)
        q = self.q()
        for b, (m, n) in enumerate(zip(self.qlens, self.kvlens)):
            s0 = int(self.start[b])
            j = np.arange(n)
            page = self.table[b].numpy()[j // self.page]
            ok = torch.from_numpy((page >= 0) & (page < self.pages))
            page = np.where(ok.numpy(), page, 0)
            pos = n - m + torch.arange(m)
            seen = (torch.arange(n) <= pos[:, None]) & ok
            if self.window:
                seen &= torch.arange(n) > pos[:, None] - self.window
            for bb, t in unseen:
                if bb == b:
                    seen[:, t] = False
            for h in range(self.heads):
                at = (page, h // group, j % self.page // 32, j % 32)
                want, wlse, size, reach = R.attend(q[s0:s0 + m, h], k[at], v[at], seen, scale)
                got, glse = out[s0:s0 + m, h].double(), lse[s0:s0 + m, h].double()
                assert torch.equal(torch.isnan(got), torch.isnan(want)), (b, h)
                ds = 2.0 ** -15 * reach[:, None]
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -15) * size + 1e-30
                off = torch.nan_to_num((got - want).abs())
                assert bool((off <= torch.nan_to_num(tol, nan=1.0)).all()), (b, h, float((off / tol).max()))
                inf = torch.isinf(wlse)
                assert torch.equal(torch.isinf(glse), inf) and bool((glse[inf] < 0).all())
                off = torch.nan_to_num((glse - wlse).abs())
                assert torch.equal(torch.isnan(glse), torch.isnan(wlse))
                assert bool((off[~inf] <= (ds[:, 0] + 2.0 ** -18 * (1 + torch.nan_to_num(wlse).abs()))[~inf]).all()), (b, h)


SHAPES = [  # qlens, kvlens, heads, kv_heads, D, page, window
    ([1], [1], 1, 1, 128, 32, 0),
    ([1, 1, 1, 1, 1], [0, 1, 31, 32, 33], 8, 1, 128, 64, 0),
    ([1, 1, 1], [95, 96, 97], 12, 3, 64, 32, 0),
    ([1, 1], [65, 300], 5, 1, 256, 128, 0),
    ([2, 1, 5, 3], [200, 0, 5, 131], 28, 4, 64, 32, 0),       # 35 rows: three row tiles
    ([5, 4], [150, 77], 12, 1, 128, 64, 0),                   # 60 rows: four
    ([3, 5], [99, 130], 7, 1, 256, 32, 0),                    # several row blocks at D = 256
    ([2, 1], [500, 333], 8, 2, 128, 64, 100),                 # a window
    ([4, 3], [64, 90], 6, 2, 64, 32, 1),                      # a window of one token
    ([7, 3], [4, 2], 4, 2, 128, 32, 0),                       # more queries than tokens: rows that see nothing
    ([40], [5], 4, 2, 64, 32, 3),
    ([1], [5003], 8, 1, 128, 256, 0),                         # split over workgroups
    ([1, 1], [4097, 2049], 3, 1, 64, 64, 0),
    ([2], [3001], 9, 1, 256, 64, 777),
    ([100], [700], 8, 2, 128, 64, 0),                         # several row blocks, split
    ([33, 70], [70, 70], 12, 4, 64, 32, 20),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("odd", [False, True])
def test_parity(shape, odd):
    announce(f"kv4_attention {shape} odd={odd}")
    c = Case(*shape, odd=odd)
    c.check(*c.run(odd_out=odd))


@pytest.mark.parametrize("D,heads,hk,m,n,window", [(64, 16, 8, 700, 720, 0), (128, 32, 8, 600, 800, 0), (128, 8, 8, 1100, 1111, 90),
                                                  (256, 16, 8, 300, 333, 0), (64, 16, 16, 2100, 2111, 0),
                                                  (128, 32, 8, 1100, 1300, 0), (128, 32, 8, 1100, 1111, 90),
                                                  (256, 16, 8, 1100, 1133, 0)])
def test_prompts(D, heads, hk, m, n, window):
    """Enough rows that every wave has its own."""
    announce(f"kv4_attention prompt {D} {heads} {hk} {m} {n} {window}")
    c = Case([m, m - 7, 1], [n, n - 13, 0], heads, hk, D, 64, window)
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_query_sizes(D):
    """Rows of tiny, huge, zero and mixed queries; scales of the cache to match."""
    c = Case([1] * 6, [40] * 6, 4, 1, D, 32)
    c.kb[:] = c.kb - 40
    f = c.flat.float()
    f[0] *= 2.0 ** 40
    f[1] *= 2.0 ** -60
    f[2] = 0
    f[3] *= 2.0 ** torch.randint(-30, 40, f[3].shape, generator=torch.Generator().manual_seed(1)).float()
    f[4] = 1.5e-38
    f[5] = 2.0 ** 39
    c.flat = f.bfloat16()
    c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores_move_the_maximum(D):
    """Scores that rise along the tokens, so that every tile moves the maximum,
    and fall, so that only the first does."""
    for sign in (1, -1):
        c = Case([1, 2], [700, 513], 4, 1, D, 64)
        c.kc[:] = 2  # all ones
        j = np.arange(c.page // 32 * 32).reshape(c.page // 32, 32)
        for b, n in enumerate(c.kvlens):
            for i, p in enumerate(c.table[b, :-(-n // c.page)].numpy()):
                c.kb[p] = (118 + sign * ((i * c.page + j) // 100))[None, :, :, None]
        c.flat = c.flat.abs()
        c.check(*c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("m", [1, 6])
def test_what_a_row_does_not_see_adds_nothing(D, m):
    """NaN scales past the tokens, before the window and after a query's own
    position: rows that see such a token are NaN, no others."""
    c = Case([m, m], [100, 64], 4, 2, D, 64, window=50)
    for b, n in enumerate(c.kvlens):
        pages = c.table[b].numpy()
        for t in [j for j in range(128) if j >= n or j < n - m + 1 - 50]:
            if t // 64 < -(-n // 64):
                c.kb[pages[t // 64], :, t % 64 // 32, t % 32] = 255
                c.vb[pages[t // 64], :, t % 64 // 32, t % 32] = 255
    out, lse = c.run()
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    c.check(out, lse)
    # a V group that only the last query of the first sequence sees
    p = c.table[0, 1]
    c.vb[p, 0, 1, 3, 1] = 255  # token 99, channels 32..63 of key head 0
    out, lse = c.run()
    want = torch.zeros(2 * m, 4, D, dtype=torch.bool)
    want[m - 1, :2, 32:64] = True
    assert torch.equal(torch.isnan(out), want)
    c.check(out, lse)
    # a K group: the whole row
    c.kb[p, 1, 1, 3, 0] = 255
    out, lse = c.run()
    want[m - 1, 2:] = True
    assert torch.equal(torch.isnan(out), want)


def test_nan_value_in_tiles_that_all_rows_see():
    c = Case([1, 3], [300, 200], 8, 1, 128, 64)
    c.vb[c.table[0, 1], 0, 0, 5, 2] = 255
    c.vb[c.table[1, 0], 0, 1, 31, 0] = 255
    out, lse = c.run()
    c.check(out, lse)
    assert int(torch.isnan(out).sum()) == 8 * 32 + 3 * 8 * 32


@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_that_are_not_finite(D):
    c = Case([2], [70], 4, 2, D, 32)
    f = c.flat.clone()
    f[0, 5], f[1, D + 1] = float("inf"), float("nan")
    c.flat = f
    out, lse = c.run()
    nan = torch.zeros(2, 4, dtype=torch.bool)
    nan[0, 0] = nan[1, 1] = True
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
    assert torch.equal(torch.isnan(lse), nan)


def test_pages_outside_the_cache_are_not_seen():
    c = Case([1, 2], [200, 160], 4, 1, 128, 32)
    c.table[0, 2], c.table[0, 5], c.table[1, 0], c.table[1, 4] = -1, c.pages, 1 << 29, -(1 << 31)
    c.check(*c.run())
    c.table[:] = -5  # nothing at all
    out, lse = c.run()
    assert not out.any() and bool((lse == -math.inf).all())


def test_lengths_outside_their_tables():
    """kv_len past the table's entries is cut, negative is none; rows of q_start
    past max_q are left alone."""
    c = Case([1, 1, 4], [64, 64, 96], 2, 1, 64, 32)
    c.table = c.table[:, :2].contiguous()
    c.kvlens = [500, -3, 64]
    out, lse = c.run(max_q=4, max_kv=64)
    c.kvlens = [64, 0, 64]
    c.check(out, lse)
    out, lse = c.run(max_q=2)
    assert bool((out[4:] == 7).all()) and bool((lse[4:] == 7).all())


def test_scale_and_bounds_that_are_not_the_lengths():
    c = Case([3, 1], [190, 40], 6, 2, 128, 64)
    c.check(*c.run(scale=0.5), scale=0.5)
    one = c.run()
    for mq, mk in ((64, 4096), (3, 100000), (3, 0), (500, 190)):
        out, lse = c.run(max_q=mq, max_kv=mk)
        c.check(out, lse)
    again = c.run()
    assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


def test_one_workspace_for_calls_of_all_sizes():
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    cases = [Case(*s) for s in SHAPES[:3] + SHAPES[11:15]]
    first = [c.run(ws) for c in cases]
    for c, f in zip(reversed(cases), reversed(first)):
        c.check(*f)
        again = c.run(ws)
        assert torch.equal(f[0], again[0]) and torch.equal(f[1], again[1])


def test_on_another_stream_and_in_a_graph():
    """One decode step of all three operators on a side stream, then captured
    and replayed on new inputs, each replay against the eager calls."""
    T, hq, hk, D, page, n = 3, 8, 2, 128, 64, 1500
    c = Case([1] * T, [n, n - 100, 7], hq, hk, D, page)
    d = lambda x: x.to(DEV)  # noqa: E731
    cache0 = d(torch.from_numpy(R.pack(c.kc, c.kb, c.vc, c.vb)))
    table, start, kv = d(c.table), d(c.start), d(torch.tensor(c.kvlens, dtype=torch.int32))
    last = torch.tensor(c.kvlens) - 1
    slots = d(c.table[torch.arange(T), last // page].long() * page + last % page)
    cs = d(torch.randn(2000, D))
    w = d(torch.ones(D, dtype=torch.bfloat16))
    pos = d(last)
    ws = torch.zeros(ar.ar_kv4_attention_workspace(T, T, 1, n, hq, hk, D), dtype=torch.uint8, device=DEV)
    qkv = torch.empty(T, hq + 2 * hk, D, dtype=torch.bfloat16, device=DEV)
    cache = cache0.clone()
    q = torch.empty(T, hq, D, dtype=torch.bfloat16, device=DEV)
    k = torch.empty(T, hk, D, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(T, hq, device=DEV)

    def step(stream=None):
        ar.ar_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hk], w, w, cs, pos, q, k, stream=stream)
        ar.ar_kv4_write(k, qkv[:, hq + hk:], slots, cache, page, stream=stream)
        ar.ar_kv4_attention(q, cache, table, start, kv, out, lse, ws, page_size=page, kv_heads=hk, max_q=1, max_kv=n, stream=stream)

    side = torch.cuda.Stream()
    inputs = [d(torch.randn(T, hq + 2 * hk, D, generator=torch.Generator().manual_seed(i)).bfloat16()) for i in range(4)]
    want = []
    for x in inputs:
        qkv.copy_(x)
        cache.copy_(cache0)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        want.append((out.clone(), lse.clone(), cache.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, (o, l, ca) in zip(inputs, want):
        qkv.copy_(x)
        cache.copy_(cache0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l) and torch.equal(cache, ca)
    qkv.copy_(inputs[0])
    cache.copy_(cache0)
    step()
    assert torch.equal(out, want[0][0])


def test_a_cache_past_4_gib():
    """Pages whose bytes lie past 2^32 (and past 2^31 tiles' bytes)."""
    D, hk, page = 256, 8, 256
    pages = 8300  # 8300 x 8 x 8 tiles of 8704 bytes: 4.6 GB
    cache = torch.zeros(pages, hk, page // 32, 34 * D, dtype=torch.uint8, device=DEV)
    assert cache.numel() > 2 ** 32
    g = torch.Generator().manual_seed(0)
    n = 300
    k, v = torch.randn(n, hk, D, generator=g).bfloat16(), torch.randn(n, hk, D, generator=g).bfloat16()
    order = [pages - 1, pages // 2 + 11]
    slots = torch.tensor([order[j // page] * page + j % page for j in range(n)])
    ar.ar_kv4_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache, page)
    c = Case([2], [n], 16, hk, D, page)
    small = R.pack(c.kc, c.kb, c.vc, c.vb)
    for i, p in enumerate(order):
        small[c.table[0, i]] = cache[p].cpu().numpy()
    c.kc, c.kb, c.vc, c.vb = R.unpack(small, D)
    c.kc, c.kb, c.vc, c.vb = (x.astype(np.int64) for x in (c.kc, c.kb, c.vc, c.vb))
    q = c.q().contiguous().to(DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 16, device=DEV)
    ws = torch.zeros(ar.ar_kv4_attention_workspace(1, 2, 2, n, 16, hk, D), dtype=torch.uint8, device=DEV)
    ar.ar_kv4_attention(q, cache, torch.tensor([order], dtype=torch.int32, device=DEV), c.start.to(DEV),
                        torch.tensor([n], dtype=torch.int32, device=DEV), out, lse, ws, page_size=page, kv_heads=hk, max_q=2, max_kv=n)
    c.check(out.cpu(), lse.cpu())
    assert np.array_equal(c.kc.shape, (c.pages, hk, page // 32, 32, D))


@pytest.mark.parametrize("D,heads,hk,m,n", [(64, 16, 8, 520, 700), (128, 32, 8, 300, 300), (256, 16, 8, 260, 333),
                                               (64, 48, 16, 1100, 1200), (128, 32, 8, 1100, 1100), (256, 16, 8, 1100, 1133)])
def test_prompts_with_nan_and_lost_pages(D, heads, hk, m, n):
    """Many rows: NaN values that some rows of a tile see, NaN past the tokens,
    pages outside the cache."""
    c = Case([m, m - 3, 2], [n, n - 5, 1], heads, hk, D, 32)
    first = n - m  # what the second query sees last
    for t, g in ((first + 1, 0), (first + 40, 1), (n - 1, 0)):
        c.vb[c.table[0, t // 32], 1, 0, t % 32, g] = 255
    c.kb[c.table[1, 1], 0, 0, 5, 0] = 255
    for b in range(2):
        p = c.table[b, (c.kvlens[b] - 1) // 32]
        c.vb[p, :, 0, (c.kvlens[b] - 1) % 32 + 1:] = 255
        c.kb[p, :, 0, (c.kvlens[b] - 1) % 32 + 1:] = 255
    c.table[0, 2], c.table[1, 0] = c.pages + 3, -1
    out, lse = c.run()
    c.check(out, lse)
    assert torch.isnan(out).any() and not torch.isnan(out).all()
