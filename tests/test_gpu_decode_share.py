"""The decode example's step, all ranks together, against the 64-bit
definitions.

Tolerance.  Keys, values and queries are taken as the step itself leaves them
(their own tests hold them to their definitions), so what is off is the
attention's output (2^-8 of itself and of its sizes, test_gpu_kv4_attention.py,
here bounded by 2^-6 of the sum of weight |v|), the product with the projection
(rounded to bf16, 2^-8) and the sum of the ranks' bf16 partial sums (2^-8): with
s the product of those sizes, 2^-6 s + 2^-7 (sum over ranks of |partial|)."""
from __future__ import annotations

import importlib.util
import pathlib

import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_util import announce

pytestmark = pytest.mark.gpu


def _example():
    path = pathlib.Path(__file__).resolve().parents[1] / "examples" / "decode_share.py"
    spec = importlib.util.spec_from_file_location("decode_share", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_of_all_ranks():
    E = _example()
    P, B, hq, hk, D, n = 4, 3, 4, 2, 64, 70
    announce(f"decode_share {P} ranks")
    layer = E.Layer(P, B, hq, hk, D, n + 2)
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda").bfloat16()

    keys = [[normal(n, hk, D) for _ in range(B)] for _ in range(P)]
    values = [[normal(n, hk, D) for _ in range(B)] for _ in range(P)]
    layer.fill(keys, values)
    for step in range(2):
        qkv = [normal(B, hq + 2 * hk, D) for _ in range(P)]
        raw = [x.clone() for x in qkv]
        sums = [x.clone() for x in layer.step(qkv)]
        assert all(torch.equal(x, sums[0]) for x in sums[1:])
        want = torch.zeros(B, layer.hidden, dtype=torch.float64)
        size, parts = want.clone(), want.clone()
        pos = torch.full((B,), n + step)
        for r in range(P):
            cs = layer.cos_sin.cpu()[pos]
            q, _ = R.norm_rope(raw[r].cpu()[:, :hq], layer.q_weight.cpu(), cs, 1e-6, False)
            got = qkv[r].cpu()[:, :hq].double()
            assert bool(((got - q).abs() <= 2.0 ** -7 * q.abs() + 2.0 ** -16).all())
            code = R.unpack(layer.cache[r].cpu().numpy(), D)
            k, v = R.values(code[0], code[1]), R.values(code[2], code[3])
            for b in range(B):
                j = np.arange(n + step + 1)
                page = layer.table[b].cpu().numpy()[j // E.PAGE]
                new = R.values(*R.quantise(qkv[r].cpu()[b, hq:hq + hk]))
                assert np.array_equal(k[page[-1], :, j[-1] % E.PAGE // 32, j[-1] % 32], new)
                o, a = torch.zeros(hq, D, dtype=torch.float64), torch.zeros(hq, D, dtype=torch.float64)
                for h in range(hq):
                    at = (page, h // (hq // hk), j % E.PAGE // 32, j % 32)
                    seen = torch.ones(1, len(j), dtype=torch.bool)
                    x, _, s, _ = R.attend(got[b, h][None], k[at], v[at], seen, D ** -0.5)
                    o[h], a[h] = x[0], s[0]
                w = layer.projection[r].cpu().double()
                part = o.reshape(-1) @ w
                want[b] += part
                parts[b] += part.abs()
                size[b] += a.reshape(-1) @ w.abs()
        off = (sums[0].cpu().double() - want).abs()
        assert bool((off <= 2.0 ** -6 * size + 2.0 ** -7 * parts).all()), float((off / size).max())
