"""CPU tests of the attention operators' boundary: refusals come before any
launch, sizes of buffers are what the header says, and the binding checks every
tensor.  Nothing here reaches a GPU."""
from __future__ import annotations

import pytest
import torch

import attention_ref as R
from allreduce_reduction_way_amd import ar

FAKE = 0x7F0000000000  # never dereferenced: every call fails its checks, or has nothing to do
MB = 1 << 20


def rows(at, ts, hs):
    return ar.ar_rows(at, ts, hs)


def norm(**kw):
    a = dict(q=rows(FAKE, 9 * 128, 128), k=rows(FAKE + 8 * 256, 9 * 128, 128), qw=FAKE + MB, kw=FAKE + 2 * MB, cs=FAKE + 3 * MB,
             pos=FAKE + 5 * MB, qo=rows(FAKE + 6 * MB, 8 * 128, 128), ko=rows(FAKE + 7 * MB, 128, 128), T=4, hq=8, hk=1, D=128, r=128,
             table=100, eps=1e-6)
    a.update(kw)
    return ar.lib().ar_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["cs"], a["pos"], a["qo"], a["ko"], a["T"], a["hq"], a["hk"],
                                    a["D"], a["r"], a["table"], a["eps"], 0, 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(hq=-1), dict(D=96), dict(D=0), dict(r=0), dict(r=144), dict(r=24), dict(table=0), dict(eps=-1.0),
    dict(eps=float("nan")), dict(qw=0), dict(kw=0), dict(cs=0), dict(pos=0), dict(qw=FAKE + MB + 1), dict(cs=FAKE + 3 * MB + 2),
    dict(pos=FAKE + 5 * MB + 4), dict(q=rows(0, 1152, 128)), dict(q=rows(FAKE + 1, 1152, 128)), dict(q=rows(FAKE, -1152, 128)),
    dict(k=rows(FAKE, 1152, -1)), dict(q=rows(FAKE, 1 << 60, 128)), dict(qo=rows(FAKE + 6 * MB, 8 * 128, 64)),
    dict(qo=rows(FAKE + 6 * MB, 0, 128))])
def test_norm_rope_refuses(kw):
    assert norm(**kw) == ar.AR_EINVAL


@pytest.mark.parametrize("kw", [
    dict(qo=rows(FAKE + 2, 9 * 128, 128)),                 # over q, shifted
    dict(qo=rows(FAKE, 9 * 128, 128), q=rows(FAKE, 9 * 128, 64)),
    dict(ko=rows(FAKE, 9 * 128, 128)),                     # keys' output over queries
    dict(qo=rows(FAKE + MB - 64, 8 * 128, 128)),           # over a weight
    dict(qo=rows(FAKE + 3 * MB + 512, 8 * 128, 128)), dict(ko=rows(FAKE + 5 * MB, 128, 128)),
    dict(ko=rows(FAKE + 6 * MB + 256, 8 * 128, 128))])     # the outputs over each other
def test_norm_rope_aliases(kw):
    assert norm(**kw) == ar.AR_EALIAS


def test_norm_rope_with_nothing_to_do():
    assert norm(T=0, q=rows(0, 0, 0), qw=0) == ar.AR_OK
    assert norm(hq=0, hk=0, q=rows(0, 0, 0), k=rows(0, 0, 0)) == ar.AR_OK


def test_norm_rope_bwd_refuses():
    L = ar.lib()
    ok = dict(gq=rows(FAKE, 1024, 128), gk=rows(FAKE + MB, 128, 128), q=rows(FAKE + 2 * MB, 1024, 128), k=rows(FAKE + 3 * MB, 128, 128),
              w=FAKE + 4 * MB, w2=FAKE + 5 * MB, cs=FAKE + 6 * MB, pos=FAKE + 8 * MB, dq=rows(FAKE + 9 * MB, 1024, 128),
              dk=rows(FAKE + 10 * MB, 128, 128), dw=FAKE + 11 * MB, dw2=FAKE + 12 * MB, ws=FAKE + 13 * MB, T=4)

    def call(**kw):
        a = {**ok, **kw}
        return L.ar_qk_norm_rope_bwd(a["gq"], a["gk"], a["q"], a["k"], a["w"], a["w2"], a["cs"], a["pos"], a["dq"], a["dk"], a["dw"],
                                     a["dw2"], a["ws"], a["T"], 8, 1, 128, 128, 100, 1e-6, 0, 0)

    for kw in (dict(T=-1), dict(dw=0), dict(dw2=0), dict(ws=0), dict(ws=FAKE + 13 * MB + 4), dict(dw=FAKE + 11 * MB + 2),
               dict(gq=rows(0, 1024, 128)), dict(dk=rows(FAKE + 10 * MB, 64, 128))):
        assert call(**kw) == ar.AR_EINVAL, kw
    for kw in (dict(dw=FAKE + 12 * MB + 8), dict(ws=FAKE + 9 * MB), dict(dw=FAKE + 4 * MB), dict(dq=rows(FAKE + MB, 1024, 128)),
               dict(dk=rows(FAKE + 2 * MB, 128, 128)), dict(dq=rows(FAKE + 10 * MB - 256, 1024, 128))):
        assert call(**kw) == ar.AR_EALIAS, kw


def test_workspaces_and_cache_sizes():
    assert ar.ar_kv4_cache_bytes(3, 2, 128, 64) == 3 * 2 * 2 * 34 * 128
    assert ar.ar_kv4_cache_bytes(0, 1, 64, 32) == 0
    for bad in ((1, 0, 128, 64), (1, 1, 96, 64), (1, 1, 128, 48), (1, 1, 128, 16), (-1, 1, 128, 64), (1 << 27, 1, 128, 32),
                (1, 1, 128, 1 << 17)):
        with pytest.raises(ar.ArError):
            ar.ar_kv4_cache_bytes(*bad)
    for bad in ((-1, 1, 1, 64), (1, -1, 1, 64), (1, 1, 1, 65)):
        with pytest.raises(ar.ArError):
            ar.ar_qk_norm_rope_bwd_workspace(*bad)
    for bad in ((-1, 1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 1, 80), (1, 1, 1, -1, 1, 1, 64),
                (1, 1, 1 << 24, 1, 128, 1, 64)):
        with pytest.raises(ar.ArError):
            ar.ar_kv4_attention_workspace(*bad)
    assert ar.ar_kv4_attention_workspace(1, 1, 1, 1, 8, 1, 128) >= 16


def kv4(fn, **kw):
    a = dict(k=rows(FAKE, 256, 128), v=rows(FAKE + MB, 256, 128), slots=FAKE + 2 * MB, cache=FAKE + 3 * MB, T=4, hk=2, D=128, pages=4,
             page=64)
    a.update(kw)
    if fn == "ar_kv4_write":
        return ar.lib().ar_kv4_write(a["k"], a["v"], a["slots"], a["cache"], a["T"], a["hk"], a["D"], a["pages"], a["page"], 0)
    return ar.lib().ar_kv4_read(a["cache"], a["slots"], a["k"], a["v"], a["T"], a["hk"], a["D"], a["pages"], a["page"], 0)


@pytest.mark.parametrize("fn", ["ar_kv4_write", "ar_kv4_read"])
def test_cache_refuses(fn):
    for kw in (dict(T=-1), dict(hk=0), dict(D=32), dict(page=33), dict(page=96), dict(pages=-1), dict(pages=1 << 26), dict(slots=0),
               dict(slots=FAKE + 2 * MB + 4), dict(cache=0), dict(cache=FAKE + 3 * MB + 8), dict(k=rows(0, 256, 128)),
               dict(v=rows(FAKE + MB + 1, 256, 128))):
        assert kv4(fn, **kw) == ar.AR_EINVAL, kw
    for kw in (dict(k=rows(FAKE + 3 * MB + 64, 256, 128)), dict(v=rows(FAKE + 3 * MB - 64, 256, 128)), dict(slots=FAKE + 3 * MB + 8)):
        assert kv4(fn, **kw) == ar.AR_EALIAS, kw
    assert kv4(fn, T=0, slots=0) == ar.AR_OK


def test_reading_into_rows_that_overlap():
    assert kv4("ar_kv4_read", k=rows(FAKE, 128, 128)) == ar.AR_EINVAL
    assert kv4("ar_kv4_read", v=rows(FAKE + 128, 256, 128)) == ar.AR_EALIAS


def attend(**kw):
    a = dict(q=rows(FAKE, 1024, 128), cache=FAKE + MB, table=FAKE + 2 * MB, ts=4, qs=FAKE + 3 * MB, kv=FAKE + 4 * MB,
             out=rows(FAKE + 5 * MB, 1024, 128), lse=FAKE + 6 * MB, ws=FAKE + 7 * MB, T=4, B=4, hq=8, hk=1, D=128, pages=8, page=64,
             per=4, mq=1, mk=256, window=0, scale=0.1)
    a.update(kw)
    return ar.lib().ar_kv4_attention(a["q"], a["cache"], a["table"], a["ts"], a["qs"], a["kv"], a["out"], a["lse"], a["ws"], a["T"],
                                     a["B"], a["hq"], a["hk"], a["D"], a["pages"], a["page"], a["per"], a["mq"], a["mk"], a["window"],
                                     a["scale"], 0)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(B=-1), dict(hq=0), dict(hk=3), dict(D=100), dict(page=40), dict(pages=-1), dict(per=-1), dict(per=1 << 30),
    dict(ts=-1), dict(mq=0), dict(mq=-1), dict(mk=-1), dict(window=-1), dict(window=1 << 31), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(qs=0), dict(kv=0), dict(lse=0), dict(ws=0), dict(table=0), dict(cache=0),
    dict(cache=FAKE + MB + 8), dict(ws=FAKE + 7 * MB + 8), dict(lse=FAKE + 6 * MB + 2), dict(qs=FAKE + 3 * MB + 1),
    dict(q=rows(0, 1024, 128)), dict(out=rows(FAKE + 5 * MB, 1024, 64)), dict(mq=1 << 24, hq=128)])
def test_attention_refuses(kw):
    assert attend(**kw) == ar.AR_EINVAL


@pytest.mark.parametrize("kw", [
    dict(out=rows(FAKE, 1024, 128)), dict(lse=FAKE + 5 * MB + 4), dict(ws=FAKE + 5 * MB), dict(lse=FAKE + MB), dict(ws=FAKE + 4 * MB),
    dict(out=rows(FAKE + 2 * MB, 1024, 128)), dict(ws=FAKE + MB), dict(lse=FAKE + 3 * MB)])
def test_attention_aliases(kw):
    assert attend(**kw) == ar.AR_EALIAS


def test_attention_with_nothing_to_do():
    assert attend(T=0, q=rows(0, 0, 0), lse=0) == ar.AR_OK
    assert attend(B=0, mq=0) == ar.AR_OK


# ------------------------------------------------------------------ the binding

def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_binding_checks_norm_rope():
    good = dict(q=_bf(4, 8, 64), k=_bf(4, 1, 64), qw=_bf(64), kw=_bf(64), cs=torch.zeros(9, 64), pos=torch.zeros(4, dtype=torch.int64))
    for kw, match in ((dict(q=_bf(4, 8, 64).float()), "bfloat16"), (dict(q=_bf(4, 512)), "shape"), (dict(k=_bf(3, 1, 64)), "shape"),
                      (dict(k=_bf(4, 1, 32)), "shape"), (dict(qw=_bf(65)), "shape"), (dict(kw=_bf(128)[::2]), "contiguous"),
                      (dict(cs=torch.zeros(9, 64).double()), "float32"), (dict(cs=torch.zeros(64, 9).t()), "contiguous"),
                      (dict(pos=torch.zeros(4, dtype=torch.int32)), "int64"), (dict(pos=torch.zeros(5, dtype=torch.int64)), "shape"),
                      (dict(q=_bf(4, 64, 8).transpose(1, 2)), "channels")):
        a = {**good, **kw}
        with pytest.raises(ValueError, match=match):
            ar.ar_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["cs"], a["pos"], stream=0)
    with pytest.raises(ValueError, match="q_out"):
        ar.ar_qk_norm_rope(*good.values(), _bf(4, 8, 128), stream=0)
    with pytest.raises(TypeError):
        ar.ar_qk_norm_rope(FAKE, *list(good.values())[1:], stream=0)
    with pytest.raises(TypeError, match="CUDA"):
        ar.ar_qk_norm_rope(*good.values(), stream=0)  # all fits, but nothing is on a GPU
    with pytest.raises(ValueError, match="workspace"):
        ar.ar_qk_norm_rope_bwd(good["q"], good["k"], *good.values(), good["q"], good["k"], torch.zeros(64), torch.zeros(64),
                               torch.zeros(8, dtype=torch.uint8), stream=0)


def test_binding_checks_the_cache():
    k, slots = _bf(4, 2, 64), torch.zeros(4, dtype=torch.int64)
    cache = torch.zeros(3, 2, 2, 34 * 64, dtype=torch.uint8)
    for args, match in (((k, _bf(4, 1, 64), slots, cache, 64), "v: shape"), ((k, k, slots[:3], cache, 64), "slots"),
                        ((k, k, slots.int(), cache, 64), "int64"), ((k, k, slots, cache, 128), "cache"),
                        ((k, k, slots, cache.int(), 64), "uint8"), ((k, k, slots, cache[:, :, ::2], 32), "contiguous")):
        with pytest.raises(ValueError, match=match):
            ar.ar_kv4_write(*args, stream=0)
        with pytest.raises(ValueError):
            ar.ar_kv4_read(args[3], args[2], args[0], args[1], args[4], stream=0)


def test_binding_checks_attention():
    i32 = torch.int32
    good = dict(q=_bf(4, 8, 64), cache=torch.zeros(3, 2, 2, 34 * 64, dtype=torch.uint8), table=torch.zeros(4, 3, dtype=i32),
                qs=torch.zeros(5, dtype=i32), kv=torch.zeros(4, dtype=i32), out=_bf(4, 8, 64), lse=torch.zeros(4, 8),
                ws=torch.zeros(1 << 20, dtype=torch.uint8))
    kw = dict(page_size=64, kv_heads=2, max_q=1, max_kv=100, stream=0)
    for bad, match in ((dict(q=_bf(4, 8, 32)), "out"), (dict(out=_bf(5, 8, 64)), "out"), (dict(lse=torch.zeros(8, 4)), "lse"),
                       (dict(lse=torch.zeros(4, 8).double()), "float32"), (dict(table=torch.zeros(4, 3).long()), "int32"),
                       (dict(table=torch.zeros(3, 4, dtype=i32).t()), "page_table"), (dict(qs=torch.zeros(4, dtype=i32)), "q_start"),
                       (dict(kv=torch.zeros(5, dtype=i32)), "kv_len"), (dict(cache=good["cache"][:, :1].contiguous()), "cache"),
                       (dict(ws=torch.zeros(8, dtype=torch.uint8)), "workspace")):
        with pytest.raises(ValueError, match=match):
            ar.ar_kv4_attention(*{**good, **bad}.values(), **kw)
    with pytest.raises(ar.ArError):
        ar.ar_kv4_attention(*good.values(), **{**kw, "max_q": -1})


# --------------------------------------------------------------- the definition

@pytest.mark.parametrize("D", [64, 128, 256])
def test_places_cover_a_tile_once(D):
    pk, pv, sk, sv = R.places(D)
    every = sorted([*pk[:, 0::2].ravel(), *pv[:, 0::2].ravel(), *sk.ravel(), *sv.ravel()])
    assert every == list(range(34 * D))
    assert (pk[:, 0::2] == pk[:, 1::2]).all() and (pv[:, 0::2] == pv[:, 1::2]).all()


def test_quantising_by_hand():
    x = torch.zeros(1, 64)
    x[0, :8] = torch.tensor([6.9, 6.0, 5.0, 3.5, 2.5, 0.25, -0.75, -7.0 / 2])
    x[0, 32:36] = torch.tensor([7.0, 1.0, 2.5, -3.0])
    code, byte = R.quantise(x)
    assert byte.tolist() == [[127, 128]]
    assert code[0, :8].tolist() == [7, 7, 6, 6, 4, 0, 10, 14]
    assert code[0, 32:36].tolist() == [6, 1, 2, 11]  # 7 / 2 = 3.5 ties to 4, 1.25 to 1
    assert R.values(code, byte)[0, 32:36].tolist() == [8.0, 1.0, 2.0, -3.0]
