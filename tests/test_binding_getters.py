"""Where the binding gets the current device and stream from."""
from types import SimpleNamespace

import pytest
import torch

import paged_kv_cascade_gb300 as pkc


def test_a_torch_without_its_internal_getters_is_asked_through_its_wrappers():
    streams = {3: SimpleNamespace(cuda_stream=0x77)}
    cuda = SimpleNamespace(current_device=lambda: 3, current_stream=lambda index: streams[index])
    device, stream = pkc._getters(SimpleNamespace(_C=SimpleNamespace(), cuda=cuda))
    assert device() == 3 and stream(3) == 0x77
    internal = SimpleNamespace(_cuda_getDevice=lambda: 1, _cuda_getCurrentRawStream=lambda index: 0x10 + index)
    device, stream = pkc._getters(SimpleNamespace(_C=internal, cuda=cuda))
    assert device() == 1 and stream(1) == 0x11


@pytest.mark.gpu
def test_both_kinds_of_getters_agree():
    torch.zeros(1, device="cuda")
    fast = pkc._getters(torch)
    plain = pkc._getters(SimpleNamespace(_C=SimpleNamespace(), cuda=torch.cuda))
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            assert fast[0]() == plain[0]() == torch.cuda.current_device()
            assert fast[1](fast[0]()) == plain[1](plain[0]()) == stream.cuda_stream
            assert pkc._stream(None) == stream.cuda_stream
