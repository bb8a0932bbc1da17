"""CPU tests: the decode example refuses more tokens than its caches hold before it
looks up a page.  Nothing here reaches a GPU."""
from __future__ import annotations

import importlib.util
import pathlib

import pytest
import torch


def _layer(room):
    path = pathlib.Path(__file__).resolve().parents[1] / "examples" / "decode_share.py"
    spec = importlib.util.spec_from_file_location("decode_share", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    layer = object.__new__(module.Layer)  # without its GPU buffers
    layer.P = layer.B = 0  # nothing to launch
    layer.hq, layer.hk, layer.room, layer.used = 4, 2, room, 0
    layer.length = torch.zeros(0, dtype=torch.int32)
    return layer


def test_a_prompt_that_does_not_fit():
    layer = _layer(70)
    with pytest.raises(ValueError, match="room for 70"):
        layer.fill([[torch.zeros(71, 2, 64)]], [[torch.zeros(71, 2, 64)]])
    layer.fill([[torch.zeros(70, 2, 64)]], [[torch.zeros(70, 2, 64)]])
    with pytest.raises(ValueError, match="71 tokens"):
        layer.step([])
    layer.fill([[torch.zeros(3, 2, 64)]], [[torch.zeros(3, 2, 64)]])
    assert layer.used == 3
