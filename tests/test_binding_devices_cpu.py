"""Tensors in host memory or on another GPU than the current one, which the library would take for addresses of
the current one: refused by the binding, before the library is reached."""
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

STREAM = types.SimpleNamespace(cuda_stream=0)


def launched(*_):
    raise AssertionError("the call reached the library")


class On:
    """A tensor as the binding looks at it, on GPU `device`."""

    def __init__(self, t, device):
        self.t, self.device = t, device

    def get_device(self):
        return self.device

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def current(monkeypatch):
    """GPU 1 is the current one, and the library fails the test."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 3)
    monkeypatch.setattr(abi, "_only", None)
    lib = types.SimpleNamespace(gdn_rope=launched, gdn_adapters_create=launched)
    monkeypatch.setattr(abi, "_lib", lib)
    monkeypatch.setattr(abi, "load_library", lambda: lib)


def refused(call, *args, **kw):
    with pytest.raises(abi.GDNError) as e:
        call(*args, **kw)
    assert e.value.name == "GDN_ERR_ARG", e.value


@pytest.mark.parametrize("device", [-1, 0, 2])
def test_adapters(current, device):
    bf = lambda *s: On(torch.zeros(*s, dtype=torch.bfloat16), device)
    scale = On(torch.ones(2), device)
    refused(abi.Adapters, bf(2, 8, 64), bf(2, 16, 8), scale)
    with pytest.raises(AssertionError):
        one = lambda *s: On(torch.zeros(*s, dtype=torch.bfloat16), 1)
        abi.Adapters(one(2, 8, 64), one(2, 16, 8), On(torch.ones(2), 1))


def test_adapters_in_host_memory(current):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    refused(abi.Adapters, bf(2, 8, 64), bf(2, 16, 8))


@pytest.mark.parametrize("device", [0, 2])
def test_rope(current, device):
    rope = types.SimpleNamespace(handle=1, d=64)
    at, q = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, 64)
    refused(abi.gdn_rope, rope, On(at, device), On(q, device), stream=STREAM)
    with pytest.raises(AssertionError):
        abi.gdn_rope(rope, On(at, 1), On(q, 1), stream=STREAM)
