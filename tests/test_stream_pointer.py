"""The current stream's handle, with and without the torch functions that give it without a stream object."""
import types

import dequant_gemv_q2_gb300 as q2


def test_current_stream(monkeypatch):
    import torch
    current = types.SimpleNamespace(cuda_stream=1234)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current)
    for have in ((), ("_cuda_getDevice",), ("_cuda_getCurrentRawStream", "_cuda_getDevice")):
        c = types.SimpleNamespace()
        if "_cuda_getDevice" in have:
            c._cuda_getDevice = lambda: 3
        if "_cuda_getCurrentRawStream" in have:
            c._cuda_getCurrentRawStream = lambda device: 5000 + device
        monkeypatch.setattr(torch, "_C", c)
        assert q2._stream_ptr(None) == (5003 if len(have) == 2 else 1234)
    assert q2._stream_ptr(types.SimpleNamespace(cuda_stream=77)) == 77
