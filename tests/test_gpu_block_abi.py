"""The operators around a block driven from plain C (tests/block_abi_check.c): raw
hipMalloc'd pointers, one stream, no PyTorch in the call path.  The results are
checked against the 64-bit definitions, with the tolerances of
test_gpu_block_norm.py, test_gpu_w4.py and test_gpu_w4_experts.py."""
from __future__ import annotations

import pathlib
import subprocess

import pytest
import torch

import attention_ref as A
import block_ref as N
import w4_ref as R
from gpu_util import announce
from test_gpu_block_norm import close as close_norm
from test_gpu_w4 import close

pytestmark = pytest.mark.gpu

EXE = pathlib.Path(__file__).resolve().parent / "block_abi_check"
T, H, P, OUT, E, I, K = 5, 320, 3, 100, 6, 96, 2


def test_plain_c_caller(tmp_path):
    if not EXE.exists():
        raise FileNotFoundError(f"{EXE} is not built: run the package build")
    g = torch.Generator().manual_seed(8)
    n = lambda *s, size=1.0: (size * torch.randn(*s, generator=g)).bfloat16()  # noqa: E731
    parts, x, post, gate, pre = n(P, T, H), n(T, H), 1 + n(H, size=0.2), n(H, size=0.5), 1 + n(H, size=0.2)
    w, router, up, down = n(OUT, H, size=H ** -0.5), n(E, H, size=H ** -0.5), n(E, 2 * I, H, size=H ** -0.5), n(E, H, I, size=I ** -0.5)
    src, dst = tmp_path / "in.bin", tmp_path / "out.bin"
    src.write_bytes(b"".join(t.view(torch.int16).numpy().tobytes() for t in (parts, x, post, gate, pre, w, router, up, down)))
    announce("block_abi_check")
    res = subprocess.run([str(EXE), str(src), str(dst)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stderr
    raw, at = bytearray(dst.read_bytes()), 0

    def take(*shape, t=torch.bfloat16):
        nonlocal at
        size = torch.Size(shape).numel()
        v = torch.frombuffer(raw, dtype=t, count=size, offset=at).reshape(shape)
        at += size * v.element_size()
        return v

    h, z, dx, dy = (take(T, H) for _ in range(4))
    dgate, dpost, dpre = (take(H, t=torch.float32) for _ in range(3))
    back, y, out, choice, weight = take(OUT, H), take(T, OUT), take(T, H), take(T, K, t=torch.int32), take(T, K, t=torch.float32)
    assert at == len(raw)
    want = N.block_norm(list(parts), x, post, gate, pre, 1.0, 1e-6)
    close_norm(h, want[0], 2.0 ** -18, "h")
    close_norm(z, want[1], 2.0 ** -18, "z")
    want = N.block_norm_grad(h, z, parts[0], x, post, gate, pre, 1.0, 1e-6)
    for got, k in ((dx, "dx"), (dy, "dy"), (dgate, "gate"), (dpost, "post"), (dpre, "pre")):
        close_norm(got, want[k], 2.0 ** -17 if got.dim() > 1 else 2.0 ** -16, k)
    values = lambda m: torch.from_numpy(A.values(*A.quantise(m)))  # noqa: E731
    assert torch.equal(back.double(), values(w))
    close(y, *R.linear(z, values(w)), "y")
    (value, size), c, p = R.experts(z, router, [values(m) for m in up], [values(m) for m in down], K, 1.5)
    assert torch.equal(choice.long(), c) and bool(((weight.double() - p).abs() <= 2.0 ** -20 * p).all())
    close(out, value, size, "out", 2.0 ** -15)
