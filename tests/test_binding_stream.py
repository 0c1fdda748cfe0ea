"""The binding's default stream is torch's current one, whether or not torch has the calls that ask for its handle
directly."""
import types

import pytest
import torch

import gated_deltanet_verify_gb300 as gdn


@pytest.fixture
def fresh(monkeypatch):
    for name in ("_torch", "_current_stream"):
        if hasattr(gdn, name):
            monkeypatch.setattr(gdn, name, None)
    return monkeypatch


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_without_the_direct_calls(fresh, missing):
    streams = iter([0, 7, 8])
    fresh.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=next(streams)))
    fresh.delattr(torch._C, missing, raising=False)
    assert gdn._stream(None) == 7 and gdn._stream(None) == 8          # the first was asked to initialise CUDA


def test_with_them(fresh):
    fresh.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=1))
    fresh.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    fresh.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    assert gdn._stream(None) == 103
    assert gdn._stream(5) == 5 and gdn._stream(types.SimpleNamespace(cuda_stream=6)) == 6


@pytest.mark.gpu
def test_on_a_device(fresh):
    torch.cuda.set_device(0)
    s = torch.cuda.Stream()
    assert gdn._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(s):
        assert gdn._stream(None) == s.cuda_stream
    assert gdn._stream(None) == torch.cuda.current_stream().cuda_stream
