"""The serving calls' choice of device and stream, without a GPU."""

import pytest
import torch

import gguf_block_quant_dequant_amd as g


def test_a_stream_of_another_device_is_refused(monkeypatch):
    class Stream:
        cuda_stream = 0x1234

        def __init__(self, device_index):
            self.device_index = device_index

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    entered = []

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            entered.append(self.what)

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(torch.cuda, "stream", Context)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x1234, raising=False)
    calls = []
    with pytest.raises(ValueError, match="device 1"):
        g._call(0, Stream(1), calls.append)
    assert not calls and not entered   # before anything changes
    own = Stream(1)
    g._call(1, own, calls.append)
    assert calls == [0x1234] and entered == [1, own]
