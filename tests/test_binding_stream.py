"""The stream that a call without one goes to."""
import types

import pytest
import torch

import edge_moe_serving_gb300 as moe


@pytest.mark.parametrize("name", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_a_torch_without_the_private_names(monkeypatch, name):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 5, raising=False)
    assert moe._s(None) == 5
    monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert moe._s(None) == 77


def test_a_given_stream_is_taken():
    assert moe._s(9) == 9 and moe._s(types.SimpleNamespace(cuda_stream=11)) == 11


@pytest.mark.gpu
def test_the_current_stream_is_taken():
    s = torch.cuda.Stream()
    assert moe._s(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):
        assert moe._s(None) == s.cuda_stream
