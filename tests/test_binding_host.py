"""The bindings' host side (no GPU needed)."""
import torch

from activation_sparse_gated_tcgen05_gb300 import twell


def test_stream_handle_without_the_raw_call(monkeypatch):
    """Where PyTorch lacks the call for a stream's raw handle, its Stream object has it."""
    class Stream:
        cuda_stream = 1234

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    assert twell._stream(None) == 1234
    assert twell._stream(Stream) == 1234 and twell._stream(77) == 77
