"""GPU parity of the norms around a block, and of their gradient, against the
64-bit definitions.

Tolerances.  One rounding of a result to bf16, half a step: 2^-8 of it.  In
binary32 before it, each step off by 2^-24 of what it adds up: sums of a row (16
channels of a lane one after another, then ten steps of a tree, so below 2^-19 of
the sum, and half of that in its root), up to seven additions of parts, and some
twenty operations, one row's sum within another's: below 2^-18 of the sizes that
the definitions return, 2^-17 backwards, where a third sum comes on top.  Gradients of
what tokens share are binary32 sums of terms with that error; a lane adds at most
one term of each 256th token, and 16 of every 64 workgroups' sums come one after
another: 2^-16 of the terms' sizes."""
from __future__ import annotations

import pytest
import torch

import block_ref as R
from allreduce_reduction_way_amd import ar
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8
EPS = 1e-5

CASES = [  # tokens, dim, parts, post, gate, pre
    (1, 1, 1, True, "token", True), (1, 7, 2, True, "shared", True), (3, 8, 1, False, "none", True), (2, 9, 3, True, "none", False),
    (5, 63, 4, False, "token", False), (4, 64, 5, True, "shared", True), (7, 513, 6, True, "token", True), (2, 1000, 7, True, "shared", True),
    (8, 5120, 8, True, "none", True), (3, 5113, 1, True, "token", True), (300, 520, 2, False, "shared", True), (2, 8192, 8, True, "token", True),
    (3, 8193, 1, True, "shared", True), (2, 8200, 8, False, "token", True), (5, 16384, 2, True, "none", True), (2, 16383, 3, True, "token", True),
    (1031, 1024, 1, True, "shared", True)]


def make(T, D, P, post, gate, pre, seed, pad=0):
    """Tensors on the CPU; rows lie `pad` elements further apart than they are long."""
    g = torch.Generator().manual_seed(seed)

    def rows(size=1.0):
        t = torch.full((T, D + pad), 3.0, dtype=torch.bfloat16)
        t[:, :D] = (size * torch.randn(T, D, generator=g) * torch.exp(0.5 * torch.randn(D, generator=g))).bfloat16()
        return t

    s = {"parts": [rows(0.5) for _ in range(P)], "x": rows(), "h_grad": rows(), "z_grad": rows() if pre else None}
    if T > 2:
        s["x"][1] = 0
        for p in s["parts"]:
            p[1] = 0  # a row of zeros
    s["post"] = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16() if post else None
    s["pre"] = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16() if pre else None
    s["gate"] = {"none": None, "shared": (0.5 * torch.randn(D, generator=g)).bfloat16(), "token": rows(0.5)}[gate]
    return s


def cut(t, D):
    return t if t is None or t.dim() == 1 else t[:, :D]


def dev(t, D):
    return None if t is None else cut(t.to(DEV), D)


def close(got, want, rel, what):
    value, size = want
    off = (got.cpu().double() - value).abs()
    tol = (BF if got.dtype == torch.bfloat16 else 0.0) * value.abs() + rel * size + 1e-30
    assert bool((off <= tol).all()), f"{what}: {float((off / tol).max())} times the tolerance"


def out_rows(T, D, pad):
    """Rows to be written, among others that must not be."""
    base = torch.full((T + 2, D + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    return base, base[1:T + 1, :D]


def untouched(base, D):
    b = base.clone()
    b[1:-1, :D] = 7.0
    return bool((b == 7.0).all())


@pytest.mark.parametrize("T,D,P,post,gate,pre", CASES)
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("scale", [1.0, -0.75])
def test_forward(T, D, P, post, gate, pre, pad, scale):
    announce(f"block_norm {T} {D} {P} {post} {gate} {pre} pad={pad}")
    s = make(T, D, P, post, gate, pre, T + D + P, pad)
    x, parts = dev(s["x"], D), [dev(p, D) for p in s["parts"]]
    weights = dict(post_weight=dev(s["post"], D), gate=dev(s["gate"], D), pre_weight=dev(s["pre"], D), residual_scale=scale, eps=EPS)
    (bh, h), (bz, z) = out_rows(T, D, pad), out_rows(T, D, pad)
    ar.ar_block_norm(parts if P > 1 else parts[0], x, h, z if pre else None, **weights)
    want = R.block_norm([cut(p, D) for p in s["parts"]], cut(s["x"], D), s["post"], cut(s["gate"], D), s["pre"], scale, EPS)
    close(h, want[0], 2.0 ** -18, "h")
    if pre:
        close(z, want[1], 2.0 ** -18, "z")
    assert untouched(bh, D) and untouched(bz, D) and (pre or bool((z == 7.0).all()))
    kept = z.clone()
    ar.ar_block_norm(parts, x, x, z if pre else None, **weights)  # in place, the same bits
    assert torch.equal(x, h) and torch.equal(z, kept)


@pytest.mark.parametrize("T,D,P,post,gate,pre", CASES)
@pytest.mark.parametrize("pad", [0, 5])
def test_gradient(T, D, P, post, gate, pre, pad):
    announce(f"block_norm_grad {T} {D} {post} {gate} {pre} pad={pad}")
    s = make(T, D, 1, post, gate, pre, T + D, pad)
    t = {k: dev(s[k], D) for k in ("x", "h_grad", "z_grad", "post", "gate", "pre")}
    y = dev(s["parts"][0], D)
    if T % 2:  # h has no other reader
        s["h_grad"] = t["h_grad"] = None
    ws = torch.zeros(ar.ar_block_norm_bwd_workspace(T, D), dtype=torch.uint8, device=DEV)
    grads = {"post": torch.full((D,), 5.0, device=DEV) if post else None, "pre": torch.full((D,), 5.0, device=DEV) if pre else None}
    (bx, dx), (by, dy), (bg, dg) = out_rows(T, D, pad), out_rows(T, D, pad), out_rows(T, D, pad)
    grads["gate"] = {"none": None, "shared": torch.full((D,), 5.0, device=DEV), "token": dg}[gate]

    def call(dx, dy, **kw):
        ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], y, t["x"], dx, dy, ws, post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                             **{"gate_grad": grads["gate"], "post_grad": grads["post"], "pre_grad": grads["pre"], **kw},
                             residual_scale=0.75, eps=EPS)

    first = None
    for _ in range(3):  # one workspace, the same bits each time
        call(dx, dy)
        got = [v.clone() for v in (dx, dy, *grads.values()) if v is not None]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = got
    want = R.block_norm_grad(cut(s["h_grad"], D), cut(s["z_grad"], D), cut(s["parts"][0], D), cut(s["x"], D), s["post"], cut(s["gate"], D), s["pre"],
                             0.75, EPS)
    close(dx, want["dx"], 2.0 ** -17, "dx")
    close(dy, want["dy"], 2.0 ** -17, "dy")
    for k, v in grads.items():
        if v is not None:
            close(v, want[k], 2.0 ** -17 if v.dim() > 1 else 2.0 ** -16, k)
    assert untouched(bx, D) and untouched(by, D) and untouched(bg, D)
    # gradients that are not wanted; dx over x and dy over y, the same bits
    call(t["x"], y, gate_grad=None, post_grad=None, pre_grad=None)
    assert torch.equal(t["x"], dx) and torch.equal(y, dy)


def test_definition_of_the_gradient_by_differences():
    """The 64-bit gradient against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g).double()  # noqa: E731
    for gate_shape in ((24,), (3, 24)):
        y, x, dh, dz = n(3, 24), n(3, 24), n(3, 24), n(3, 24)
        post, pre, gate = 1 + 0.2 * n(24), 1 + 0.2 * n(24), n(*gate_shape)
        got = R.block_norm_grad(dh, dz, y, x, post, gate, pre, 0.75, EPS)

        def loss(y, x, post, gate, pre):
            (h, _), (z, _) = R.block_norm([y], x, post, gate, pre, 0.75, EPS)
            return float((h * dh).sum() + (z * dz).sum())

        at = (y, x, post, gate, pre)
        for _ in range(6):
            d, e = [n(*v.shape) for v in at], 1e-5
            num = (loss(*(v + e * w for v, w in zip(at, d))) - loss(*(v - e * w for v, w in zip(at, d)))) / (2 * e)
            want = sum(float((got[k][0] * w).sum()) for k, w in zip(("dy", "dx", "post", "gate", "pre"), d))
            assert abs(num - want) < 1e-6 * (1 + abs(num))


def test_a_token_with_infinities_and_nan_is_alone():
    T, D = 5, 1032
    announce("block_norm with infinities")
    s = make(T, D, 2, True, "token", True, 11)
    clean = [dev(p, D) for p in s["parts"]]
    dirty = [p.clone() for p in clean]
    dirty[0][1, 5], dirty[1][3, 1031] = float("nan"), float("inf")
    kw = dict(post_weight=dev(s["post"], D), gate=dev(s["gate"], D), pre_weight=dev(s["pre"], D), eps=EPS)
    got = []
    for parts in (clean, dirty):
        h, z = torch.empty(T, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
        ar.ar_block_norm(parts, dev(s["x"], D), h, z, **kw)
        got.append((h, z))
    for a, b in zip(*got):
        assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]]) and not bool(torch.isfinite(a).logical_not().any())
        assert bool(torch.isnan(b[1]).all()) and bool(torch.isnan(b[3, 1031]))


def test_no_tokens():
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    e = z(0, 64)
    ar.ar_block_norm(e, e, e, z(0, 64), pre_weight=z(64))
    ws = torch.zeros(ar.ar_block_norm_bwd_workspace(0, 64), dtype=torch.uint8, device=DEV)
    d = [torch.full((64,), 5.0, device=DEV) for _ in range(3)]
    ar.ar_block_norm_bwd(e, e, e, e, z(0, 64), z(0, 64), ws, post_weight=z(64), gate=z(64), pre_weight=z(64), gate_grad=d[0], post_grad=d[1],
                         pre_grad=d[2])
    assert not any(bool(v.any()) for v in d)


@pytest.mark.parametrize("T,D,P", [(8200, 4104, 1), (2100, 8192, 8), (2100, 16384, 2)])
def test_past_128_mib(T, D, P):
    """Rows that are streamed past the caches; the definition on the GPU."""
    announce(f"large block_norm {T} {D} {P}")
    assert 2 * T * D * (P + 3) > 128 << 20
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    parts, x, gate, post, pre = [n(T, D) for _ in range(P)], n(T, D), n(T, D), n(D), n(D)
    h, z = torch.empty_like(x), torch.empty_like(x)
    ar.ar_block_norm(parts, x, h, z, post_weight=post, gate=gate, pre_weight=pre, eps=EPS)
    pick = torch.cat([torch.arange(40), torch.randint(0, T, (80,)), torch.arange(T - 40, T)]).to(DEV)
    want = R.block_norm([p[pick].cpu() for p in parts], x[pick].cpu(), post.cpu(), gate[pick].cpu(), pre.cpu(), 1.0, EPS)
    close(h[pick], want[0], 2.0 ** -18, "h")
    close(z[pick], want[1], 2.0 ** -18, "z")
    ws = torch.zeros(ar.ar_block_norm_bwd_workspace(T, D), dtype=torch.uint8, device=DEV)
    dx, dy, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dpost, dpre = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    dh, dz = n(T, D), n(T, D)
    ar.ar_block_norm_bwd(dh, dz, parts[0], x, dx, dy, ws, post_weight=post, gate=gate, pre_weight=pre, gate_grad=dg, post_grad=dpost,
                         pre_grad=dpre, eps=EPS)
    sums = {"post": torch.zeros(D, dtype=torch.float64), "pre": torch.zeros(D, dtype=torch.float64)}
    sizes = {k: v.clone() for k, v in sums.items()}
    for at in range(0, T, 1024):
        r = slice(at, at + 1024)
        w = R.block_norm_grad(dh[r], dz[r], parts[0][r], x[r], post, gate[r], pre, 1.0, EPS)
        for got, k in ((dx, "dx"), (dy, "dy"), (dg, "gate")):
            close(got[r], (w[k][0].cpu(), w[k][1].cpu()), 2.0 ** -17, k)
        for k in sums:
            sums[k] += w[k][0].cpu()
            sizes[k] += w[k][1].cpu()
    for got, k in ((dpost, "post"), (dpre, "pre")):
        close(got, (sums[k], sizes[k]), 2.0 ** -16, k)


@pytest.mark.parametrize("T,D", [(4096, 7168), (1500, 6145), (1500, 6144), (3000, 8192), (4096, 1024), (5000, 256), (2000, 1025), (700, 2048), (2100, 2560),
                                 (300, 9000), (1, 5), (40, 7)])
def test_nothing_past_the_workspace_is_written(T, D):
    """Each rule's number of workgroups with sums of their own, in a workspace of the size asked for."""
    announce(f"block_norm_grad workspace {T} {D}")
    g = torch.Generator(device=DEV).manual_seed(T + D)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    size, guard = ar.ar_block_norm_bwd_workspace(T, D), 32 << 20
    ws = torch.full((size + guard,), 255, dtype=torch.uint8, device=DEV)
    y, x, dh, dz, gate, post, pre = n(T, D), n(T, D), n(T, D), n(T, D), n(D), n(D), n(D)
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    grads = [torch.empty(D, device=DEV) for _ in range(3)]
    ar.ar_block_norm_bwd(dh, dz, y, x, dx, dy, ws[:size], post_weight=post, gate=gate, pre_weight=pre, gate_grad=grads[0], post_grad=grads[1],
                         pre_grad=grads[2], eps=EPS)
    assert bool((ws[size:] == 255).all())
    want = R.block_norm_grad(dh, dz, y, x, post, gate, pre, 1.0, EPS)
    for k, v in (("dx", dx), ("dy", dy), ("gate", grads[0]), ("post", grads[1]), ("pre", grads[2])):
        close(v, tuple(w.cpu() for w in want[k]), 2.0 ** -17 if v.dim() > 1 else 2.0 ** -16, k)


@pytest.mark.parametrize("D", [264, 7000, 9000, 16384])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_gradient_in_place_of_what_it_reads(D, post, pre):
    """dx and dy over each of the rows, all gradients wanted: as apart from them."""
    T = 37
    announce(f"block_norm_grad in place {D} {post} {pre}")
    s = make(T, D, 1, post, "shared", pre, D)
    ws = torch.zeros(ar.ar_block_norm_bwd_workspace(T, D), dtype=torch.uint8, device=DEV)
    names = ["h_grad", "x", "y"] + (["z_grad"] if pre else [])

    def call(at_x, at_y):
        t = {k: dev(s[k], D) for k in ("x", "h_grad", "z_grad", "post", "gate", "pre")}
        t["y"] = dev(s["parts"][0], D)
        dx = t[at_x] if at_x else torch.empty_like(t["x"])
        dy = t[at_y] if at_y else torch.empty_like(t["x"])
        grads = [torch.full((D,), 5.0, device=DEV) for _ in range(3)]
        ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], t["y"], t["x"], dx, dy, ws, post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                             gate_grad=grads[0], post_grad=grads[1] if post else None, pre_grad=grads[2] if pre else None, eps=EPS)
        return dx, dy, *grads

    want = call(None, None)
    for at_x in names:
        for at_y in names:
            if at_x != at_y:
                assert all(torch.equal(a, b) for a, b in zip(call(at_x, at_y), want)), (at_x, at_y)


@pytest.mark.parametrize("D", [1000, 8200])
def test_rows_far_apart(D):
    """Strides past 2^31 elements."""
    announce(f"block_norm with long strides {D}")
    T, far = 3, (1 << 30) + 12345
    s = make(T, D, 2, True, "token", True, D)

    def spread(t):
        base = torch.empty(far * (T - 1) + D, dtype=torch.bfloat16, device=DEV)
        v = base.as_strided((T, D), (far, 1))
        if t is not None:
            v.copy_(t[:, :D])
        return v

    parts, x, gate, h, z = [spread(p) for p in s["parts"]], spread(s["x"]), spread(s["gate"]), spread(None), spread(None)
    w = dict(post_weight=dev(s["post"], D), gate=gate, pre_weight=dev(s["pre"], D), eps=EPS)
    ar.ar_block_norm(parts, x, h, z, **w)
    want = R.block_norm(s["parts"], s["x"], s["post"], s["gate"], s["pre"], 1.0, EPS)
    close(h, want[0], 2.0 ** -18, "h")
    close(z, want[1], 2.0 ** -18, "z")
    ws = torch.zeros(ar.ar_block_norm_bwd_workspace(T, D), dtype=torch.uint8, device=DEV)
    dg, sums = spread(None), [torch.empty(D, device=DEV) for _ in range(2)]
    h.copy_(s["h_grad"])
    z.copy_(s["z_grad"])
    ar.ar_block_norm_bwd(h, z, parts[0], x, x, parts[1], ws, **w, gate_grad=dg, post_grad=sums[0], pre_grad=sums[1])
    want = R.block_norm_grad(s["h_grad"], s["z_grad"], s["parts"][0], s["x"], s["post"], s["gate"], s["pre"], 1.0, EPS)
    for got, k in ((x, "dx"), (parts[1], "dy"), (dg, "gate")):
        close(got, want[k], 2.0 ** -17, k)
    for got, k in zip(sums, ("post", "pre")):
        close(got, want[k], 2.0 ** -16, k)


@pytest.mark.parametrize("T,D", [(1, 5), (2, 7), (1, 6144), (2, 6144), (3, 6144), (1, 6152), (2, 6152), (1, 8192), (2, 100), (3, 100), (1, 8200), (32, 8200), (33, 8200)])
@pytest.mark.parametrize("wanted", [(True, True, True), (False, True, False), (True, False, True)])
def test_gradients_of_a_few_tokens(T, D, wanted):
    """Sums of one workgroup, and of a few, where some are not wanted."""
    announce(f"block_norm_grad few {T} {D} {wanted}")
    s = make(T, D, 1, True, "shared", True, T + D)
    t = {k: dev(s[k], D) for k in ("x", "h_grad", "z_grad", "post", "gate", "pre")}
    y, dx, dy = dev(s["parts"][0], D), torch.empty_like(t["x"]), torch.empty_like(t["x"])
    ws = torch.full((ar.ar_block_norm_bwd_workspace(T, D),), 255, dtype=torch.uint8, device=DEV)
    base = torch.full((3, D + 2), 5.0, device=DEV)
    grads = [base[i, 1:-1] if w else None for i, w in enumerate(wanted)]
    ar.ar_block_norm_bwd(t["h_grad"], t["z_grad"], y, t["x"], dx, dy, ws, post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                         gate_grad=grads[0], post_grad=grads[1], pre_grad=grads[2], eps=EPS)
    want = R.block_norm_grad(s["h_grad"], s["z_grad"], s["parts"][0], s["x"], s["post"], s["gate"], s["pre"], 1.0, EPS)
    close(dx, want["dx"], 2.0 ** -17, "dx")
    close(dy, want["dy"], 2.0 ** -17, "dy")
    for i, k in enumerate(("gate", "post", "pre")):
        if wanted[i]:
            close(base[i, 1:-1], want[k], 2.0 ** -16, k)
            base[i, 1:-1] = 5.0
    assert bool((base == 5.0).all())


@pytest.mark.parametrize("D", [6136, 6144, 6145, 6152, 8191, 8192])
@pytest.mark.parametrize("P", [1, 4, 5])
def test_forward_around_the_change_of_lanes(D, P):
    announce(f"block_norm lanes {D} {P}")
    T = 3
    s = make(T, D, P, True, "shared", True, D + P)
    h, z = torch.empty(T, D, dtype=torch.bfloat16, device=DEV), torch.empty(T, D, dtype=torch.bfloat16, device=DEV)
    ar.ar_block_norm([dev(p, D) for p in s["parts"]], dev(s["x"], D), h, z, post_weight=dev(s["post"], D), gate=dev(s["gate"], D),
                     pre_weight=dev(s["pre"], D), eps=EPS)
    want = R.block_norm([cut(p, D) for p in s["parts"]], s["x"], s["post"], s["gate"], s["pre"], 1.0, EPS)
    close(h, want[0], 2.0 ** -18, "h")
    close(z, want[1], 2.0 ** -18, "z")
