"""CPU tests: calls beyond the attention operators' documented sizes are refused
before any launch.  Addresses are never dereferenced."""
from __future__ import annotations

from allreduce_reduction_way_amd import ar

BASE, FAR = 0x100000000000, 1 << 42


def rows(i, ts, hs):
    return ar.ar_rows(BASE + i * FAR, ts, hs)


def test_norms():
    def call(T, hq=1, hk=1, D=64):
        at = [BASE + (10 + i) * FAR for i in range(4)]
        return ar.lib().ar_qk_norm_rope(rows(0, hq * D, D), rows(1, hk * D, D), *at, rows(2, hq * D, D), rows(3, hk * D, D), T, hq, hk, D, D,
                                        100, 1e-6, 0, 0)

    assert call(1 << 24) == call(1 << 28) == call((1 << 28) + 1) == ar.AR_EINVAL
    assert call(1, hq=65537) == call(1, hk=65537) == ar.AR_EINVAL


def test_cache():
    def call(T, hk=1, D=64, pages=1 << 20):
        return ar.lib().ar_kv4_write(rows(0, hk * D, D), rows(1, hk * D, D), BASE + 10 * FAR, BASE + 20 * FAR, T, hk, D, pages, 32, 0)

    assert call((1 << 28) + 1) == call(1 << 26, hk=8) == call(1, hk=65537) == ar.AR_EINVAL


def test_attention():
    def call(T=4, B=4, hq=8, hk=1, D=64, mq=1):
        return ar.lib().ar_kv4_attention(rows(0, hq * D, D), BASE + 10 * FAR, BASE + 11 * FAR, 4, BASE + 12 * FAR, BASE + 13 * FAR,
                                         rows(1, hq * D, D), BASE + 14 * FAR, BASE + 15 * FAR, T, B, hq, hk, D, 8, 64, 4, mq, 256, 0, 0.1, 0)

    for kw in (dict(B=(1 << 20) + 1), dict(T=(1 << 28) + 1), dict(mq=(1 << 24) + 1), dict(hq=1 << 15), dict(hq=8192, hk=8192),
               dict(mq=1 << 18, hq=8192), dict(B=1 << 20, hk=8, T=1 << 20)):
        assert call(**kw) == ar.AR_EINVAL, kw
