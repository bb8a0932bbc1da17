"""Plain 64-bit definitions of the products with 4-bit weights, on the CPU, written
from the formulas of include/ar.h.  Results come with their sizes: what they add up
from, in magnitudes."""
from __future__ import annotations

import numpy as np
import torch

import attention_ref as A


def tile_bytes(n_in):
    c = -(-n_in // 128)
    return 1024 * c + 256 * (-(-c // 4))


def places(n_out, n_in):
    """Where the codes (n_out, n_in) and scales (n_out, n_in / 32) lie: tile, byte."""
    r, k, g = np.arange(n_out)[:, None], np.arange(n_in)[None], np.arange(n_in // 32)[None]
    c = -(-n_in // 128)
    code = 1024 * (k // 128) + (16 * (k % 128 // 32) + r % 16) * 16 + k % 32 // 2
    scale = 1024 * c + 256 * (g // 16) + (16 * (g % 4) + r % 16) * 4 + g // 4 % 4
    return r // 16, code, scale


def pack(code, byte):
    """Codes (n_out, n_in) and scale bytes (n_out, n_in / 32) as tiles; what is named by no place stays 0."""
    n, k = code.shape
    tile, pc, ps = places(n, k)
    out = np.zeros((-(-n // 16), tile_bytes(k)), dtype=np.uint8)
    out[tile, pc[:, 0::2]] = code[:, 0::2] | code[:, 1::2] << 4
    out[tile, ps] = byte
    return out


def unpack(packed, n_out, n_in):
    tile, pc, ps = places(n_out, n_in)
    return packed[tile, pc] >> (np.arange(n_in) % 2 * 4) & 15, packed[tile, ps]


def values(packed, n_out, n_in):
    """(n_out, n_in) in 64 bits."""
    return torch.from_numpy(A.values(*unpack(packed, n_out, n_in)))


def random_weights(n_out, n_in, g, size=1.0):
    """Packed weights of about that size, every code among them, and their values."""
    code = torch.randint(0, 16, (n_out, n_in), generator=g, dtype=torch.uint8).numpy()
    byte = torch.randint(-2, 1, (n_out, n_in // 32), generator=g).numpy() + 126 + int(np.floor(np.log2(size)))
    packed = pack(code, byte.astype(np.uint8))
    return torch.from_numpy(packed), values(packed, n_out, n_in)


def linear(x, w):
    x = x.double()
    return x @ w.T, x.abs() @ w.abs().T


def choose(logits, k):
    """logits (T, E) in binary32: indices (T, k), from the largest; of two alike the lower."""
    return torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]


def experts(x, router, gate_up, down, k, scale):
    """gate_up, down: lists of values in 64 bits.  (out, size), choice, weight."""
    x = x.double()
    logits = (x @ router.double().T).float()
    choice = choose(logits, k)
    taken = logits.gather(1, choice).double()
    weight = torch.softmax(taken, 1) * scale
    out, size = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    for e in range(router.shape[0]):
        rows, at = (choice == e).nonzero(as_tuple=True)
        if not len(rows):
            continue
        (both, sizes), half = linear(x[rows], gate_up[e]), gate_up[e].shape[0] // 2
        g, u, gs, us = both[:, :half], both[:, half:], sizes[:, :half], sizes[:, half:]
        s = g * torch.sigmoid(g)
        a = s * u
        w = weight[rows, at][:, None]
        out[rows] += w * (a @ down[e].T)
        # silu' is 1.1 at most
        size[rows] += w.abs() * ((1.1 * gs * u.abs() + us * s.abs() + a.abs()) @ down[e].abs().T)
    return (out, size), choice, weight
