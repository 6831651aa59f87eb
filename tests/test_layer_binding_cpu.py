"""Checks of the layer's Python side that need no GPU."""

import types

import pytest
import torch

import bit_ptq_vla_amd as q
from bit_ptq_vla_amd.workload import DecoderLayer


def test_decoder_layer_refuses_lengths_behind_its_rotary_table():
    layer = DecoderLayer.__new__(DecoderLayer)
    layer.rope = torch.zeros((64, 16))
    with pytest.raises(ValueError, match="rotary table of 64 positions"):
        layer.step(torch.zeros((1, 16)), torch.zeros((1, 16)), types.SimpleNamespace(max_kv=65))


def test_stream_handle_without_the_raw_accessor(monkeypatch):
    monkeypatch.setattr(q, "_raw_stream", None, raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1234))
    assert q._stream(torch.device("cuda", 0)) == 1234
