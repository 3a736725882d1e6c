"""Sizes that do not fit the library's int32, or whose index arithmetic would not: refused, not cut off."""
import ctypes
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from gated_deltanet_recurrent_gb300 import build as gbuild

STREAM = types.SimpleNamespace(cuda_stream=0)


class Sized:
    """A tensor of that shape, of which nothing but its attributes is there."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def stride(self, i=None):
        s = [1]
        for x in reversed(self.shape[1:]):
            s.insert(0, s[0] * x)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x1000


def refused(name, call, *args, **kw):
    with pytest.raises(abi.GDNError) as e:
        call(*args, **kw)
    assert e.value.name == name, e.value


@pytest.fixture
def nothing_launched(monkeypatch):
    def launched(*_):
        raise AssertionError("the call reached the library")
    lib = types.SimpleNamespace(gdn_rope=launched, gdn_adapters_create=launched,
                                gdn_kv_pages_grow=launched)
    monkeypatch.setattr(abi, "_lib", lib)
    monkeypatch.setattr(abi, "load_library", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(abi, "_only", 0)


@pytest.mark.parametrize("a,b", [((2 ** 32 + 1, 8, 64), (2 ** 32 + 1, 16, 8)),
                                 ((2, 8, 2 ** 32 + 64), (2, 16, 8)), ((2, 8, 64), (2, 2 ** 32 + 16, 8))])
def test_adapters(nothing_launched, a, b):
    scale = Sized(a[0], dtype=torch.float32)
    refused("GDN_ERR_UNSUPPORTED", abi.Adapters, Sized(*a), Sized(*b), scale)


def test_rope(nothing_launched):
    n = 2 ** 32 + 3
    refused("GDN_ERR_SIZE", abi.gdn_rope, types.SimpleNamespace(handle=1, d=64),
            Sized(n, dtype=torch.int32), Sized(n, 2, 64), stream=STREAM)


def test_pages(nothing_launched):
    n = 2 ** 32 + 3
    kv = types.SimpleNamespace(handle=1, page_table=torch.full((4, 3), -1, dtype=torch.int32),
                               desc=types.SimpleNamespace(n_slots=4, n_pages=6))
    book = abi.KVPages(kv)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    refused("GDN_ERR_SIZE", abi.gdn_kv_pages_grow, kv, book, i32(0), i32(0), i32(0, 3),
            rows=Sized(n, dtype=torch.int64), stream=STREAM)
    refused("GDN_ERR_SIZE", abi.gdn_kv_pages_grow, kv, book, i32(0), i32(0), i32(0, 3), n, stream=STREAM)


@pytest.mark.parametrize("hidden", [2 ** 30 + 1, 2 ** 31 - 1, 2 ** 31 - 64])
def test_hidden(hidden):
    gbuild.build()
    lib = abi.load_library()
    desc, out = abi.gdn_adapters_desc(1, 1, hidden, 8, 0), ctypes.c_void_p()
    st = lib.gdn_adapters_create(ctypes.byref(desc), 0x1000, 0, 0x2000, 8, 0x3000, ctypes.byref(out))
    assert abi.STATUS[st] == "GDN_ERR_UNSUPPORTED" and out.value is None
