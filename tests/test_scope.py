"""The binding's handling of devices and streams around a call, with stand-ins for CUDA (no GPU needed)."""
import pytest
import torch

import precision_attention_forward_b200 as lp


class _Device:
    """Stands in for torch.cuda.device: records what is entered and left."""
    log = []

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.log.append(("in", self.device.index))

    def __exit__(self, *exc):
        self.log.append(("out", self.device.index))


class _Stream:
    cuda_stream = 77

    def __init__(self, device):
        self.device = device


@pytest.fixture
def on_device_0(monkeypatch):
    _Device.log = []
    monkeypatch.setattr(torch.cuda, "device", _Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: _Stream(torch.device("cuda", 1)))


def test_a_refused_stream_leaves_the_current_device_as_it_was(on_device_0):
    with pytest.raises(ValueError, match="stream"):
        with lp._Scope(torch.device("cuda", 1), _Stream(torch.device("cuda", 0))):
            raise AssertionError("entered")
    assert _Device.log == [("in", 1), ("out", 1)] or not _Device.log


def test_a_call_on_another_device_goes_there_and_back(on_device_0):
    with lp._Scope(torch.device("cuda", 1), _Stream(torch.device("cuda", 1))) as sc:
        assert sc.handle == 77
    assert _Device.log == [("in", 1), ("out", 1)]
    with lp._Scope(torch.device("cuda", 0), None) as sc:  # no stream given: the current one
        assert sc.handle == 0
    assert len(_Device.log) == 2
