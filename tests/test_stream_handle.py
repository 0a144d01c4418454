"""The stream that the binding hands to the library, with and without torch's own raw call."""
import types

import torch

import bf16_forward_attention_gb300 as attn


class _Tensor:
    device = torch.device("cuda", 3)

    @staticmethod
    def get_device():
        return 3


def test_raw_call(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    assert attn._stream_of(_Tensor) == 103


def test_public_call_where_there_is_no_raw_one(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device: types.SimpleNamespace(cuda_stream=200 + device.index))
    assert attn._stream_of(_Tensor) == 203
