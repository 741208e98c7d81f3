"""The stream a call goes to, on the host."""
import types

import torch

from sparse_linear_layers_group_amd import bitlinear as bl


def test_current_stream_without_the_private_name(monkeypatch):
    monkeypatch.setattr(bl, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert bl._stream(None) == 77


def test_current_stream_by_its_handle(monkeypatch):
    monkeypatch.setattr(bl, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert bl._stream(None) == 1003


def test_given_handle():
    assert bl._stream(55) == 55 and bl._stream(0) == 0
