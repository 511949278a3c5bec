"""The stream handle that every binding passes on, without a GPU."""
import types

import torch

from chunk_scheduled_communication_gb300 import syn


def test_given_streams():
    assert syn._stream(7) == 7
    assert syn._stream(types.SimpleNamespace(cuda_stream=9)) == 9


def test_current_stream_through_public_functions_alone(monkeypatch):
    """A torch without its private functions for it."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=11))
    assert syn._stream(None) == 11


def test_current_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 20 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    assert syn._stream(None) == 23
