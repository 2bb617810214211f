"""Where the binding takes the current stream's handle from, without a GPU."""
import types

import pytest

import structured_sparse_gemm_nm_amd as nm

torch = pytest.importorskip("torch")


def test_stream_without_the_private_call(monkeypatch):
    # a torch that lacks the private symbol is asked through its public interface
    asked = []
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device: asked.append(device) or types.SimpleNamespace(cuda_stream=0x5EED))
    device = torch.device("cuda", 3)
    assert nm._stream_ptr(device) == 0x5EED and asked == [device]


def test_stream_of_the_tensors_device(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    assert nm._stream_ptr(torch.device("cuda", 2)) == 102
