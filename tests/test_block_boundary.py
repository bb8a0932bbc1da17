"""CPU tests of the boundary of the operators around a block: refusals come before
any launch, sizes of buffers are what the header says, and the binding checks every
tensor.  Nothing here reaches a GPU."""
from __future__ import annotations

import pytest
import torch

from allreduce_reduction_way_amd import ar

FAKE = 0x7F0000000000  # never dereferenced: every call fails its checks, or has nothing to do
MB = 1 << 20


def rows(at, ts):
    return ar.ar_rows(at, ts, -77)  # the stride of heads is not looked at


def ptrs(*at):
    p = ar.ar_ptrs()
    for i, a in enumerate(at):
        p.p[i] = a
    return p


# ------------------------------------------------------------------------- norms

def norm(**kw):
    a = dict(parts=ptrs(FAKE, FAKE + MB), ps=256, P=2, x=rows(FAKE + 2 * MB, 256), post=FAKE + 3 * MB, gate=rows(FAKE + 4 * MB, 256),
             pre=FAKE + 5 * MB, h=rows(FAKE + 6 * MB, 256), z=rows(FAKE + 7 * MB, 256), T=4, D=200, scale=1.0, eps=1e-6)
    a.update(kw)
    return ar.lib().ar_block_norm(a["parts"], a["ps"], a["P"], a["x"], a["post"], a["gate"], a["pre"], a["h"], a["z"], a["T"], a["D"], a["scale"],
                                  a["eps"], 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(D=0), dict(D=-8), dict(D=16385), dict(T=1 << 21), dict(P=0), dict(P=9), dict(eps=-1.0), dict(eps=float("nan")),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(parts=ptrs(FAKE, 0)), dict(parts=ptrs(FAKE, FAKE + MB + 1)), dict(ps=-256),
    dict(x=rows(0, 256)), dict(x=rows(FAKE + 2 * MB + 1, 256)), dict(x=rows(FAKE + 2 * MB, -1)), dict(x=rows(FAKE + 2 * MB, 1 << 60)),
    dict(post=FAKE + 3 * MB + 1), dict(pre=FAKE + 5 * MB + 1), dict(gate=rows(FAKE + 4 * MB + 1, 256)), dict(gate=rows(FAKE + 4 * MB, -8)),
    dict(h=rows(0, 256)), dict(h=rows(FAKE + 6 * MB, 199)), dict(h=rows(FAKE + 6 * MB, 0)), dict(z=rows(0, 256)), dict(z=rows(FAKE + 7 * MB, 100))])
def test_norm_refuses(kw):
    assert norm(**kw) == ar.AR_EINVAL


@pytest.mark.parametrize("kw", [
    dict(h=rows(FAKE, 256)), dict(h=rows(FAKE + MB + 8, 256)), dict(h=rows(FAKE + 2 * MB + 2, 256)),  # over parts, over x but shifted
    dict(h=rows(FAKE + 2 * MB, 264)),                                                               # over x, another stride
    dict(z=rows(FAKE + 2 * MB, 256)), dict(z=rows(FAKE, 256)), dict(h=rows(FAKE + 4 * MB, 256)), dict(z=rows(FAKE + 4 * MB, 256)),
    dict(h=rows(FAKE + 3 * MB, 256)), dict(z=rows(FAKE + 5 * MB + 64, 256)), dict(z=rows(FAKE + 6 * MB + 1024, 256)),
    dict(h=rows(FAKE + 4 * MB + 256, 256), gate=rows(FAKE + 4 * MB, 0))])
def test_norm_aliases(kw):
    assert norm(**kw) == ar.AR_EALIAS


def test_norm_with_nothing_to_do():
    assert norm(T=0, x=rows(0, 0), parts=ptrs(), h=rows(0, 0)) == ar.AR_OK


def test_rows_beside_each_other_are_not_refused_for_sharing():
    """h beside z in every token: only the missing eps refuses the call."""
    assert norm(h=rows(FAKE + 6 * MB, 512), z=rows(FAKE + 6 * MB + 512, 512), P=9) == ar.AR_EINVAL
    assert norm(h=rows(FAKE + 6 * MB, 512), z=rows(FAKE + 6 * MB + 256, 512)) == ar.AR_EALIAS


def bwd(**kw):
    a = dict(dh=rows(FAKE, 256), dz=rows(FAKE + MB, 256), y=rows(FAKE + 2 * MB, 256), x=rows(FAKE + 3 * MB, 256), post=FAKE + 4 * MB,
             gate=rows(FAKE + 5 * MB, 256), pre=FAKE + 6 * MB, dx=rows(FAKE + 7 * MB, 256), dy=rows(FAKE + 8 * MB, 256),
             dg=rows(FAKE + 9 * MB, 256), dpost=FAKE + 10 * MB, dpre=FAKE + 11 * MB, ws=FAKE + 12 * MB, T=4, D=200, scale=1.0, eps=1e-6)
    a.update(kw)
    return ar.lib().ar_block_norm_bwd(a["dh"], a["dz"], a["y"], a["x"], a["post"], a["gate"], a["pre"], a["dx"], a["dy"], a["dg"], a["dpost"],
                                      a["dpre"], a["ws"], a["T"], a["D"], a["scale"], a["eps"], 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(D=0), dict(D=16385), dict(T=(1 << 28) + 1), dict(eps=-1.0), dict(scale=float("nan")), dict(ws=0), dict(ws=FAKE + 12 * MB + 8),
    dict(dh=rows(FAKE + 1, 256)), dict(dz=rows(0, 256)), dict(y=rows(0, 256)), dict(x=rows(0, 256)), dict(x=rows(FAKE + 3 * MB, -1)),
    dict(post=FAKE + 4 * MB + 1), dict(pre=FAKE + 6 * MB + 1), dict(dx=rows(0, 256)), dict(dx=rows(FAKE + 7 * MB, 199)),
    dict(dy=rows(FAKE + 8 * MB, 0)), dict(dg=rows(FAKE + 9 * MB, 100)), dict(dpost=FAKE + 10 * MB + 2), dict(dpre=FAKE + 11 * MB + 2),
    dict(gate=rows(FAKE + 5 * MB, 0), dg=rows(FAKE + 9 * MB + 2, 0))])
def test_norm_bwd_refuses(kw):
    assert bwd(**kw) == ar.AR_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dx=rows(FAKE + 8 * MB, 256)), dict(dx=rows(FAKE + 2, 256)), dict(dy=rows(FAKE + 2 * MB, 264)), dict(dx=rows(FAKE + 5 * MB, 256)),
    dict(dg=rows(FAKE + 5 * MB, 256)), dict(dg=rows(FAKE + 7 * MB, 256)), dict(dg=rows(FAKE, 256)), dict(dx=rows(FAKE + 4 * MB, 256)),
    dict(dpost=FAKE + 11 * MB + 400), dict(dpost=FAKE + 4 * MB), dict(dpre=FAKE + 7 * MB), dict(ws=FAKE + 3 * MB), dict(ws=FAKE + 10 * MB),
    dict(ws=FAKE + 9 * MB), dict(gate=rows(FAKE + 5 * MB, 0), dg=rows(FAKE + 5 * MB, 0)), dict(gate=rows(FAKE + 5 * MB, 0), dg=rows(FAKE + 10 * MB, 0))])
def test_norm_bwd_aliases(kw):
    assert bwd(**kw) == ar.AR_EALIAS


def test_norm_bwd_workspace():
    for bad in ((-1, 8), (1, 0), (1, 16385)):
        with pytest.raises(ar.ArError):
            ar.ar_block_norm_bwd_workspace(*bad)
    tokens, dims = [0, 1, 2, 255, 256, 257, 1000, 1 << 20], [1, 7, 8, 100, 5120, 8191, 8192, 8193, 16384]
    for d in dims:
        sizes = [ar.ar_block_norm_bwd_workspace(t, d) for t in tokens]
        assert sizes == sorted(sizes) and all(s >= 12 * d and s % 16 == 0 for s in sizes)
    for t in tokens:
        sizes = [ar.ar_block_norm_bwd_workspace(t, d) for d in dims]
        assert sizes == sorted(sizes)


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_binding_checks_norm():
    good = dict(parts=[_bf(4, 64), _bf(4, 64)], x=_bf(4, 64), h=_bf(4, 64), z=_bf(4, 64))
    kw = dict(post_weight=_bf(64), gate=_bf(4, 64), pre_weight=_bf(64), stream=0)
    for bad, match in ((dict(x=_bf(4, 64).float()), "bfloat16"), (dict(x=_bf(4, 8, 8)), "dimensions"), (dict(h=_bf(5, 64)), "h: shape"),
                       (dict(z=_bf(4, 63)), "z: shape"), (dict(z=None), "together"), (dict(pre_weight=None), "together"),
                       (dict(parts=[]), "1 to 8"), (dict(parts=[_bf(4, 64)] * 9), "1 to 8"), (dict(parts=[_bf(4, 64), _bf(4, 65)]), "parts: shape"),
                       (dict(parts=[_bf(4, 64), _bf(4, 128)[:, :64]]), "one stride"), (dict(parts=(_bf(4, 128)[:, ::2],)), "contiguous"),
                       (dict(gate=_bf(63)), "gate: shape"), (dict(gate=_bf(1, 64)), "gate: shape"), (dict(gate=_bf(64)[None].expand(4, 64)), "one gate"),
                       (dict(post_weight=_bf(65)), "post_weight"), (dict(pre_weight=_bf(128)[::2]), "contiguous")):
        a = {**good, **kw, **bad}
        with pytest.raises(ValueError, match=match):
            ar.ar_block_norm(**a)
    for bad in (dict(parts=3), dict(parts=[FAKE]), dict(x=None), dict(h=FAKE)):
        with pytest.raises(TypeError):
            ar.ar_block_norm(**{**good, **kw, **bad})
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_block_norm(**good, **kw)  # all fits, but nothing is on a GPU
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_block_norm(_bf(4, 64), _bf(4, 64), _bf(4, 64), stream=0)


def test_binding_checks_norm_bwd():
    f = torch.zeros(64)
    good = dict(h_grad=_bf(4, 64), z_grad=_bf(4, 64), y=_bf(4, 64), x=_bf(4, 64), dx=_bf(4, 64), dy=_bf(4, 64),
                workspace=torch.zeros(4 * 3 * 64 * 4, dtype=torch.uint8))
    kw = dict(post_weight=_bf(64), gate=_bf(64), pre_weight=_bf(64), gate_grad=f, post_grad=f, pre_grad=f, stream=0)
    for bad, match in ((dict(h_grad=_bf(3, 64)), "h_grad"), (dict(z_grad=None), "together"), (dict(pre_weight=None, pre_grad=None), "together"),
                       (dict(y=_bf(4, 32)), "y: shape"), (dict(dx=_bf(4, 64).float()), "dx"), (dict(workspace=torch.zeros(8)), "workspace"),
                       (dict(gate=None), "no gate"), (dict(gate=_bf(4, 64)), "gate_grad"), (dict(gate_grad=_bf(4, 64)), "gate_grad"),
                       (dict(post_weight=None), "no post_weight"), (dict(post_grad=f.double()), "float32"),
                       (dict(z_grad=None, pre_weight=None), "no pre_weight")):
        with pytest.raises(ValueError, match=match):
            ar.ar_block_norm_bwd(**{**good, **kw, **bad})
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_block_norm_bwd(**good, **kw)
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_block_norm_bwd(**{**good, "h_grad": None}, **kw)


def test_a_gradient_that_would_be_lost_is_refused():
    x = _bf(4, 64).requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        ar.ar_block_norm([_bf(4, 64)], x, _bf(4, 64), stream=0)
    with pytest.raises(ValueError, match="requires a gradient"):
        ar.ar_block_norm([_bf(4, 64), x], _bf(4, 64), _bf(4, 64), stream=0)
    with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):
        ar.ar_block_norm([_bf(4, 64), x], _bf(4, 64), _bf(4, 64), stream=0)


# --------------------------------------------------------------- weights of 4 bits

def test_w4_bytes():
    assert ar.ar_w4_bytes(16, 128) == 1024 + 256
    assert ar.ar_w4_bytes(17, 544) == 2 * (5 * 1024 + 2 * 256)
    assert ar.ar_w4_bytes(1, 32) == 1280
    assert ar.ar_w4_bytes(1 << 24, 1 << 20) == (1 << 20) * ((1 << 13) * 1024 + (1 << 11) * 256)
    for bad in ((0, 128), (-1, 128), (16, 0), (16, 33), (16, 16), (16, -32), ((1 << 24) + 1, 32), (16, (1 << 20) + 32)):
        with pytest.raises(ar.ArError):
            ar.ar_w4_bytes(*bad)


@pytest.mark.parametrize("fn", ["pack", "unpack"])
def test_w4_pack_refuses(fn):
    def call(**kw):
        a = dict(w=FAKE, rs=160, packed=FAKE + 64 * MB, n=40, k=160)
        a.update(kw)
        args = (a["w"], a["rs"], a["packed"]) if fn == "pack" else (a["packed"], a["w"], a["rs"])
        return getattr(ar.lib(), f"ar_w4_{fn}")(*args, a["n"], a["k"], 0)

    for kw in (dict(w=0), dict(w=FAKE + 1), dict(rs=-160), dict(packed=0), dict(packed=FAKE + 64 * MB + 8), dict(n=0), dict(k=40), dict(k=0),
               dict(n=1 << 24, k=1 << 14, rs=1 << 14, w=FAKE, packed=FAKE + (1 << 45))):
        assert call(**kw) == ar.AR_EINVAL, kw
    for kw in (dict(packed=FAKE + 160), dict(w=FAKE + 64 * MB + 512)):
        assert call(**kw) == ar.AR_EALIAS, kw
    if fn == "unpack":
        assert call(rs=159) == ar.AR_EINVAL


def test_w4_linear_refuses():
    def call(**kw):
        a = dict(x=rows(FAKE, 160), w=FAKE + MB, out=rows(FAKE + 2 * MB, 40), T=4, n=40, k=160)
        a.update(kw)
        return ar.lib().ar_w4_linear(a["x"], a["w"], a["out"], a["T"], a["n"], a["k"], 0)

    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(n=0), dict(k=150), dict(x=rows(0, 160)), dict(x=rows(FAKE + 1, 160)), dict(x=rows(FAKE, -1)),
               dict(w=0), dict(w=FAKE + MB + 8), dict(out=rows(0, 40)), dict(out=rows(FAKE + 2 * MB, 39)), dict(out=rows(FAKE + 2 * MB, 0))):
        assert call(**kw) == ar.AR_EINVAL, kw
    for kw in (dict(out=rows(FAKE, 160)), dict(out=rows(FAKE + MB, 40)), dict(out=rows(FAKE + MB + 1280 * 3 - 2, 40), k=128, x=rows(FAKE, 128))):
        assert call(**kw) == ar.AR_EALIAS, kw
    assert call(T=0, x=rows(0, 0), w=0) == ar.AR_OK


def test_w4_experts_refuses():
    def call(**kw):
        a = dict(x=rows(FAKE, 160), r=FAKE + MB, gu=FAKE + 2 * MB, dn=FAKE + 4 * MB, out=rows(FAKE + 6 * MB, 160), c=FAKE + 7 * MB, w=FAKE + 8 * MB,
                 ws=FAKE + 9 * MB, T=4, H=160, I=96, E=8, k=3, scale=1.0)
        a.update(kw)
        return ar.lib().ar_w4_experts(a["x"], a["r"], a["gu"], a["dn"], a["out"], a["c"], a["w"], a["ws"], a["T"], a["H"], a["I"], a["E"], a["k"],
                                      a["scale"], 0)

    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(H=0), dict(H=150), dict(I=0), dict(I=100), dict(I=(1 << 19) + 32), dict(E=0), dict(E=513),
               dict(k=0), dict(k=9), dict(k=17, E=40), dict(scale=float("nan")), dict(scale=float("inf")), dict(x=rows(0, 160)), dict(x=rows(FAKE + 1, 160)),
               dict(r=0), dict(r=FAKE + MB + 1), dict(gu=0), dict(gu=FAKE + 2 * MB + 8), dict(dn=0), dict(dn=FAKE + 4 * MB + 4),
               dict(out=rows(0, 160)), dict(out=rows(FAKE + 6 * MB, 159)), dict(c=0), dict(c=FAKE + 7 * MB + 2), dict(w=0), dict(w=FAKE + 8 * MB + 1),
               dict(ws=0), dict(ws=FAKE + 9 * MB + 8)):
        assert call(**kw) == ar.AR_EINVAL, kw
    for kw in (dict(out=rows(FAKE, 160)), dict(out=rows(FAKE + MB, 160)), dict(c=FAKE + 2 * MB), dict(w=FAKE + 4 * MB + 64), dict(ws=FAKE + 16),
               dict(c=FAKE + 8 * MB + 4), dict(c=FAKE + 6 * MB), dict(ws=FAKE + 6 * MB), dict(w=FAKE + 9 * MB + 4096), dict(ws=FAKE + 3 * MB + 512 * 1024)):
        assert call(**kw) == ar.AR_EALIAS, kw
    assert call(T=0, x=rows(0, 0), r=0) == ar.AR_OK


def test_w4_experts_workspace_never_falls():
    for bad in ((-1, 64, 64, 4, 2), (1, 65, 64, 4, 2), (1, 64, 63, 4, 2), (1, 64, 64, 0, 1), (1, 64, 64, 4, 5), (1, 64, 64, 513, 2), (1, 64, 64, 64, 17)):
        with pytest.raises(ar.ArError):
            ar.ar_w4_experts_workspace(*bad)
    axes = ([0, 1, 2, 63, 64, 65, 1000], [32, 512, 7168], [32, 96, 1024], [16, 64, 512], [1, 2, 8, 16])
    import itertools
    for n in range(5):
        for rest in itertools.product(*(a for i, a in enumerate(axes) if i != n)):
            sizes = [ar.ar_w4_experts_workspace(*rest[:n], v, *rest[n:]) for v in axes[n]]
            assert sizes == sorted(sizes), (n, rest)


def test_binding_checks_w4():
    u8 = torch.uint8
    w, packed = _bf(40, 160), torch.zeros(3, ar.ar_w4_bytes(16, 160), dtype=u8)
    for fn in (lambda w, p: ar.ar_w4_pack(w, p, stream=0), lambda w, p: ar.ar_w4_unpack(p, w, stream=0)):
        for bad, match in ((dict(w=w.float()), "bfloat16"), (dict(w=_bf(40, 4, 40)), "dimensions"), (dict(w=_bf(160, 40).t()), "contiguous"),
                           (dict(p=packed[:2]), "packed: shape"), (dict(p=packed[:, 1:]), "packed: shape"), (dict(p=packed.int()), "uint8")):
            with pytest.raises(ValueError, match=match):
                fn(**{"w": w, "p": packed, **bad})
        with pytest.raises(TypeError, match="CUDA"):
            fn(w, packed)
        with pytest.raises(ar.ArError):
            fn(_bf(40, 50), packed)
    x, out = _bf(4, 160), _bf(4, 40)
    for bad, match in (((x.float(), packed, out), "bfloat16"), ((x, packed, _bf(5, 40)), "out: shape"), ((x, packed, _bf(4, 49)), "packed: shape"),
                       ((_bf(4, 320)[:, ::2], packed, out), "contiguous"), ((_bf(4, 288), packed, out), "packed: shape"), ((x, packed, out.view(160)), "dim")):
        with pytest.raises(ValueError, match=match):
            ar.ar_w4_linear(*bad, stream=0)
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_w4_linear(x, packed, out, stream=0)
    with pytest.raises(ar.ArError):
        ar.ar_w4_linear(_bf(4, 33), packed, out, stream=0)


def test_binding_checks_experts():
    u8, H, I, E, k, T = torch.uint8, 160, 96, 8, 3, 4
    good = dict(x=_bf(T, H), router=_bf(E, H), gate_up=torch.zeros(E, 2 * I // 16, ar.ar_w4_bytes(16, H), dtype=u8),
                down=torch.zeros(E, H // 16, ar.ar_w4_bytes(16, I), dtype=u8), out=_bf(T, H), choice=torch.zeros(T, k, dtype=torch.int32),
                weight=torch.zeros(T, k), workspace=torch.zeros(ar.ar_w4_experts_workspace(T, H, I, E, k), dtype=u8))
    for bad, match in ((dict(x=_bf(T, 192)), "router: shape"), (dict(router=_bf(7, H)), "gate_up: shape"), (dict(router=_bf(E, 2 * H)[:, ::2]), "contiguous"),
                       (dict(gate_up=good["gate_up"][:, :4]), "down: shape|gate_up"), (dict(down=good["down"][:, :9]), "down: shape"), (dict(out=_bf(T, 32)), "out: shape"),
                       (dict(choice=torch.zeros(T, k)), "int32"), (dict(choice=torch.zeros(3, k, dtype=torch.int32)), "choice: shape"),
                       (dict(weight=torch.zeros(T, 2)), "weight: shape"), (dict(workspace=torch.zeros(64, dtype=u8)), "workspace"),
                       (dict(gate_up=good["gate_up"][0]), "dimensions")):
        with pytest.raises(ValueError, match=match):
            ar.ar_w4_experts(**{**good, **bad}, stream=0)
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_w4_experts(**good, stream=0)
    with pytest.raises(ar.ArError):
        ar.ar_w4_experts(**{**good, "choice": torch.zeros(T, 9, dtype=torch.int32), "weight": torch.zeros(T, 9)}, stream=0)
    x = _bf(T, H).requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        ar.ar_w4_experts(**{**good, "x": x}, stream=0)
