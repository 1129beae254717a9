"""cache_device_status on the host: which stream it waits for, and which device's word it reads (a fake library; no GPU)."""
import ctypes
import types

import pytest
import torch

import bf16_attention_forward_gb300 as attn


class Device:
    """torch.cuda.device as a record."""
    current, log = 0, []

    def __init__(self, index):
        self.index = index

    def __enter__(self):
        self.before, Device.current = Device.current, self.index

    def __exit__(self, *_):
        Device.current = self.before


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def get(stream, site):
        seen.append((Device.current, stream.value if isinstance(stream, ctypes.c_void_p) else stream))
        ctypes.cast(site, ctypes.POINTER(ctypes.c_int32))[0] = 22
        return 1

    fake = types.SimpleNamespace(attn_cache_get_device_status=get)
    monkeypatch.setattr(attn, "load", lambda: fake)
    monkeypatch.setattr(attn, "_lib", fake)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Device.current, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream(0x50, Device.current))
    return seen


def stream(handle, index):
    return types.SimpleNamespace(cuda_stream=handle, device_index=index, device=torch.device("cuda", index))


def test_of_a_stream_on_another_device(calls):
    assert attn.cache_device_status(stream(0x70, 3)) == (1, 22)
    assert calls == [(3, 0x70)] and Device.current == 0


def test_of_the_current_stream_and_of_one_on_the_current_device(calls):
    assert attn.cache_device_status() == (1, 22)
    assert attn.cache_device_status(stream(0x60, 0)) == (1, 22)
    assert calls == [(0, 0x50), (0, 0x60)]


def test_of_a_stream_by_its_handle(calls):
    # as the four calls take it
    assert attn.cache_device_status(0x80) == (1, 22)
    assert calls == [(0, 0x80)]
