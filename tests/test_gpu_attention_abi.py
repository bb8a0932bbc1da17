"""The attention operators driven from plain C (tests/attention_abi_check.c):
raw hipMalloc'd pointers, one stream, no PyTorch in the call path.  The results
are checked against the 64-bit definitions, with the tolerances of
test_gpu_norm_rope.py and test_gpu_kv4_attention.py."""
from __future__ import annotations

import pathlib
import subprocess

import numpy as np
import pytest
import torch

import attention_ref as R
from gpu_util import announce

pytestmark = pytest.mark.gpu

EXE = pathlib.Path(__file__).resolve().parent / "attention_abi_check"
T, HQ, HK, D = 70, 4, 2, 64


def test_plain_c_caller(tmp_path):
    if not EXE.exists():
        raise FileNotFoundError(f"{EXE} is not built: run the package build")
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(T, HQ + 2 * HK, D, generator=g).bfloat16()
    angle = 6.3 * torch.rand(T, D // 2, generator=g, dtype=torch.float64)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    src, dst = tmp_path / "in.bin", tmp_path / "out.bin"
    src.write_bytes(qkv.view(torch.int16).numpy().tobytes() + cs.numpy().tobytes())
    announce("attention_abi_check")
    res = subprocess.run([str(EXE), str(src), str(dst)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    raw = dst.read_bytes()
    sizes = [2 * T * HQ * D, 2 * T * HK * D, 2 * T * HK * D, 2 * T * HK * D, 2 * T * HQ * D, 4 * T * HQ, 4 * D]
    assert len(raw) == sum(sizes)
    parts, at = [], 0
    for n in sizes:
        parts.append(bytearray(raw[at:at + n]))
        at += n
    q, k, ko, vo, out = (torch.frombuffer(p, dtype=torch.bfloat16).reshape(T, -1, D) for p in parts[:5])
    lse, dw = torch.frombuffer(parts[5], dtype=torch.float32).reshape(T, HQ), torch.frombuffer(parts[6], dtype=torch.float32)
    ones = torch.ones(D)
    for x, got in ((qkv[:, :HQ], q), (qkv[:, HQ:HQ + HK], k)):
        want, size = R.norm_rope(x, ones, cs, 1e-6, False)
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all())
    for x, got in ((k, ko), (qkv[:, HQ + HK:], vo)):
        assert np.array_equal(got.double().numpy(), R.values(*R.quantise(x)))
    _, _, wantw, sizew = R.norm_rope_grad(qkv[:, :HQ], qkv[:, :HQ], ones, cs, 1e-6, False)
    assert bool(((dw.double() - wantw).abs() <= 2.0 ** -16 * sizew).all())
    seen = torch.tril(torch.ones(T, T, dtype=torch.bool))
    for h in range(HQ):
        want, wlse, size, reach = R.attend(q[:, h], ko[:, h // 2].double().numpy(), vo[:, h // 2].double().numpy(), seen, 0.125)
        ds = 2.0 ** -15 * reach[:, None]
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * ds + 2.0 ** -15) * size
        assert bool(((out[:, h].double() - want).abs() <= tol).all())
        assert bool(((lse[:, h].double() - wlse).abs() <= ds[:, 0] + 2.0 ** -18 * (1 + wlse.abs())).all())
