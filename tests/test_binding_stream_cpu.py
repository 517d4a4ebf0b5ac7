"""Which stream a call goes to: the one it is given, else torch's current one,
also on a torch build without the raw query."""
import types

import torch

import block_top_sparse_kin_b200 as kin


def test_a_given_stream():
    assert kin._stream(7) == 7 and kin._stream(0) == 0
    assert kin._stream(types.SimpleNamespace(cuda_stream=11)) == 11


def test_the_current_stream(monkeypatch):
    monkeypatch.setattr(kin, "_current_device", lambda: 3)
    monkeypatch.setattr(kin, "_current_stream", lambda device: 100 + device)
    assert kin._stream(None) == 103
    monkeypatch.setattr(kin, "_current_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=42))
    assert kin._stream(None) == 42
