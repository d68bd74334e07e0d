"""Which stream a call without one takes (no GPU): torch's current one, by
whatever torch offers, with torch's own message where it has no CUDA."""
import types

import pytest
import torch

from sparsely_gated_mixture_gb300 import binding as B


def without_private_calls(monkeypatch):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)


def test_a_torch_without_the_raw_handle(monkeypatch):
    without_private_calls(monkeypatch)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=77 + (device or 0)))
    assert B._stream(None) in (77, 78)


def test_a_torch_without_cuda(monkeypatch):
    without_private_calls(monkeypatch)

    def refuse(*_):
        raise AssertionError("Torch not compiled with CUDA enabled")
    monkeypatch.setattr(torch.cuda, "current_device", refuse)
    monkeypatch.setattr(torch.cuda, "current_stream", refuse)
    with pytest.raises(AssertionError, match="not compiled with CUDA"):
        B._stream(None)


def test_the_raw_handle_is_the_current_devices(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device,
                        raising=False)
    assert B._stream(None) == 1003


def test_given_streams_need_no_torch(monkeypatch):
    without_private_calls(monkeypatch)
    assert B._stream(0) == 0 and B._stream(5) == 5
    assert B._stream(types.SimpleNamespace(cuda_stream=9)) == 9
