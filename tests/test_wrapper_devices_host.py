"""Streams and workspaces of another device are refused by the wrappers of the
operators of a training step, before anything is launched.  No GPU: the
stream is a stand-in."""

import pytest
import torch

from moe_layer_router_amd import layer as L


class _Stream:
    def __init__(self, handle=0, device="cuda:0"):
        self.device = torch.device(device)


def test_stream_of_another_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert L._on(torch.device("cuda:1"), _Stream(device="cuda:1")).device.index == 1
    assert L._on(torch.device("cuda:1"), 1234).device.index == 1           # a handle: of the tensors' device
    with pytest.raises(ValueError, match="stream"):
        L._on(torch.device("cuda:0"), _Stream(device="cuda:1"))


def test_workspace_of_another_device():
    ws = L.Workspace("cpu")
    assert L._scratch(ws, torch.device("cpu"), 1000).numel() == 1000
    assert L._scratch(ws, torch.device("cpu"), 10) is ws.buf
    assert L._scratch(None, torch.device("cpu"), 10).device == torch.device("cpu")
    with pytest.raises(ValueError, match="workspace"):
        L._scratch(ws, torch.device("cuda:0"), 1000)
