"""A given workspace has to be contiguous memory of its inputs' device: an expanded tensor's element count says
nothing about the memory behind it.  (On the CPU: the checks come before any call, and the tensors are stand-ins that
carry what the checks read.)"""
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4


class OnDevice:
    """A tensor's checks as on device `dev`."""

    def __init__(self, t, dev=0):
        self.t, self.dev, self.is_cuda = t, dev, True
        self.dtype, self.shape, self.device = t.dtype, t.shape, t.device

    def get_device(self):
        return self.dev

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as they would be made, none made."""
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: (made.append(name), 64 if name.endswith("bytes") else 0)[1]
    monkeypatch.setattr(fp4, "lib", Lib)
    monkeypatch.setattr(fp4, "_stream", lambda t: 0)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: torch.zeros(t.shape, dtype=t.dtype))
    return made


def attention(ws):
    i32 = lambda *s: OnDevice(torch.ones(*s, dtype=torch.int32))  # noqa: E731
    cache = fp4.KV4Cache(OnDevice(torch.zeros(2 * 16 * 2 * 68, dtype=torch.uint8)), 2, 16, 2, 64)
    return fp4.kv4_attention(OnDevice(torch.zeros(1, 4, 64, dtype=torch.bfloat16)), cache, i32(1, 2), i32(1), ws=ws)


def linear(ws):
    w = fp4.Block8(8, 32, fp4.FP4_BLOCK_SQUARE, "cpu")
    w.codes = OnDevice(w.codes)
    return fp4.block8_linear_forward(OnDevice(torch.zeros(4, 32)), w, ws=ws)


def backward(ws):
    w = fp4.Block8(32, 8, fp4.FP4_BLOCK_SQUARE, "cpu")
    w.codes = OnDevice(w.codes)
    return fp4.block8_linear_backward(OnDevice(torch.zeros(4, 8)), w, None, ws=ws)


@pytest.mark.parametrize("call,name", [(attention, "fp4_kv4_attention"), (linear, "fp4_block8_linear"),
                                       (backward, "fp4_block8_backward")])
def test_workspaces(call, name, calls):
    byte = torch.zeros(1, dtype=torch.uint8)
    for bad in (OnDevice(byte.expand(1 << 20)), OnDevice(torch.zeros(1 << 12, dtype=torch.uint8)[::2]),
                OnDevice(torch.zeros(1 << 12, dtype=torch.uint8), dev=1), torch.zeros(1 << 12, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            call(bad)
    assert name not in calls
    call(OnDevice(torch.zeros(1 << 12, dtype=torch.uint8)))
    assert name in calls
