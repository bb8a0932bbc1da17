"""GPU parity of weights of 4 bits: packing, and products of tokens with them,
against the 64-bit definitions.

Tolerances.  Codes, scales and values are exact.  A product's terms are exact in
binary32 (8 bits times 2 bits); a sum has up to 32 terms in an instruction, up to
64 instructions one after another and up to eight waves' sums, each adding 2^-24 of
the terms' magnitudes: 2^-17 of those, and one rounding to bf16, half a step:
2^-8 of the result."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as A
import w4_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


def close(got, value, size, what, rel=2.0 ** -17):
    off = (got.cpu().double() - value).abs()
    tol = BF * value.abs() + rel * size + 1e-30
    assert bool((off <= tol).all()), f"{what}: {float((off / tol).max())} times the tolerance"


@pytest.mark.parametrize("N,K", [(1, 32), (16, 128), (5, 96), (17, 160), (33, 512), (100, 544), (48, 2080), (1, 8192), (1000, 64)])
@pytest.mark.parametrize("pad", [0, 3])
def test_pack_and_unpack(N, K, pad):
    announce(f"w4_pack {N} {K} pad={pad}")
    g = torch.Generator().manual_seed(N + K)
    w = torch.full((N, K + pad), 9.0, dtype=torch.bfloat16)
    w[:, :K] = (torch.randn(N, K, generator=g) * torch.exp(3 * torch.randn(N, 1, generator=g))).bfloat16()
    w[0, :32] = 0
    w[-1, :32] *= 2.0 ** -118   # subnormal scales of the group, and below
    if N > 4:
        w[1, K - 1], w[2, 3], w[3, 0] = float("nan"), float("inf"), -float("inf")
        w[4, :32] = 3.0e38
    want = R.pack(*A.quantise(w[:, :K]))
    packed = torch.full((want.shape[0] + 2, want.shape[1]), 77, dtype=torch.uint8, device=DEV)
    assert packed.shape[1] == ar.ar_w4_bytes(16, K)
    d = w.to(DEV)[:, :K]
    ar.ar_w4_pack(d, packed[1:-1])
    got = packed.cpu().numpy()
    assert (got[0] == 77).all() and (got[-1] == 77).all()
    named = np.zeros(want.shape, dtype=bool)
    tile, pc, ps = R.places(N, K)
    named[tile, pc] = True
    named[tile, ps] = True
    assert np.array_equal(got[1:-1][named], want[named])
    codes = np.zeros(want.shape, dtype=bool)
    codes[:, :1024 * -(-K // 128)] = True
    assert not got[1:-1][codes & ~named].any()  # codes past the matrix
    back = torch.full((N + 2, K + pad), 9.0, dtype=torch.bfloat16, device=DEV)
    ar.ar_w4_unpack(packed[1:-1], back[1:-1, :K])
    b = back.cpu()
    exact = R.values(want, N, K)
    assert torch.equal(torch.isnan(b[1:-1, :K]), torch.isnan(exact))
    assert torch.equal(torch.nan_to_num(b[1:-1, :K].double()), torch.nan_to_num(exact))
    b[1:-1, :K] = 9.0
    assert bool((b == 9.0).all())


LINEAR = [  # tokens, n_in, n_out
    (1, 32, 1), (1, 64, 16), (1, 1024, 5120), (2, 96, 33), (7, 160, 100), (16, 512, 48), (17, 640, 47), (31, 1056, 130), (33, 2080, 65),
    (48, 256, 1000), (64, 1184, 500), (65, 544, 129), (130, 416, 70), (200, 96, 16), (1, 8192, 300), (3, 4064, 20000), (5, 256, 40000),
    (20, 320, 33000), (60, 288, 34001)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("pad", [0, 3])
def test_linear(T, K, N, pad):
    announce(f"w4_linear {T} {K} {N} pad={pad}")
    g = torch.Generator().manual_seed(T + K + N)
    packed, w = R.random_weights(N, K, g, K ** -0.5)
    x = torch.full((T, K + pad), 3.0, dtype=torch.bfloat16)
    x[:, :K] = torch.randn(T, K, generator=g).bfloat16()
    out = torch.full((T + 2, N + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    dx, dw = x.to(DEV)[:, :K], packed.to(DEV)
    ar.ar_w4_linear(dx, dw, out[1:-1, :N])
    value, size = R.linear(x[:, :K], w)
    close(out[1:-1, :N], value, size, "out")
    first = out.clone()
    out[1:-1, :N] = 5.0
    ar.ar_w4_linear(dx, dw, out[1:-1, :N])
    assert torch.equal(out, first)  # the same bits each time
    out[1:-1, :N] = 7.0
    assert bool((out == 7.0).all())


def test_what_lies_past_a_row_is_not_taken():
    """Infinities beside the rows of x, a token of NaN, and weights of NaN."""
    announce("w4_linear with NaN beside it")
    T, K, N = 5, 160, 40
    g = torch.Generator().manual_seed(1)
    packed, w = R.random_weights(N, K, g)
    x = torch.full((T, 512), float("inf"), dtype=torch.bfloat16)
    x[:, 100:100 + K] = torch.randn(T, K, generator=g).bfloat16()
    x[3, 107] = float("nan")
    bad = packed.clone()
    tile, _, ps = R.places(N, K)
    bad[tile[20, 0], ps[20, 2]] = 255
    out = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    ar.ar_w4_linear(x.to(DEV)[:, 100:100 + K], bad.to(DEV), out)
    nan = torch.isnan(out).cpu()
    assert bool(nan[3].all()) and bool(nan[:, 20].all())
    nan[3], nan[:, 20] = False, False
    assert not bool(nan.any())
    value, size = R.linear(x[:, 100:100 + K], w)
    keep = [0, 1, 2, 4]
    rest = [n for n in range(N) if n != 20]
    close(out[keep][:, rest], value[keep][:, rest], size[keep][:, rest], "out")


def test_no_tokens():
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(1, ar.ar_w4_bytes(16, 64), dtype=torch.uint8, device=DEV)
    ar.ar_w4_linear(z, w, torch.zeros(0, 5, dtype=torch.bfloat16, device=DEV))
