"""The committed counters and traces of the all-reduce kernels are of the sources as
they are: a change to those kernels, or to the headers that they are built from,
comes with counters recorded again, or bench.py reports no traffic."""
from __future__ import annotations

import re

import pytest

import bench

RECORDED = sorted(p.name for p in bench.PROFILES.glob("*.md") if re.search(r"[Kk]ernel source hash", p.read_text()))


def test_the_headline_reports_its_traffic():
    got = bench.traffic_from_profiles("write_bcast_440x5120_p8", 72089600)
    assert got is not None and 0.99 < got / 72089600 < 1.05


@pytest.mark.parametrize("name", RECORDED)
def test_profiles_are_of_these_sources(name):
    line = re.search(r"[Kk]ernel source hash.*", (bench.PROFILES / name).read_text()).group(0)
    hashes = re.findall(r"`([0-9a-f]{16})`", line)
    now = {bench.kernel_source_hash(), bench.kernel_source_hash(bench.PACKET_SOURCES)}
    assert hashes and hashes[0] in now, name
    if len(hashes) > 1:  # reduce, packet and probe kernels
        assert set(hashes[:2]) == now, name
