"""How the binding finds the current stream and device (CPU only: torch's side is faked)."""
import torch

import pose_retrieved_kv_b200 as P

L = P._lib


class _Stream:
    cuda_stream = 0x5EED


def test_current_stream_is_asked_of_torch_s_public_calls(monkeypatch):
    """Without torch's private shortcut the public way gives the stream."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name)
    if hasattr(L, "_raw_stream"):
        monkeypatch.setattr(L, "_raw_stream", None)
    assert L._stream(None) == 0x5EED
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    assert L._device() == 3


def test_the_shortcut_gives_the_stream_of_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(L, "_raw_stream", lambda device: 1000 + device)
    assert L._stream(None) == 1003


def test_no_device_is_looked_for_before_cuda_is_in_use(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: False)
    assert L._device() == 0
