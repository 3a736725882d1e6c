"""What the page calls refuse before any launch, at the C entries and in the binding."""
import ctypes
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from gated_deltanet_recurrent_gb300 import build as gbuild

STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return abi.load_library()


def test_a_null_cache_fails_cleanly(lib):
    book = abi.gdn_kv_pages(0x1000, 0x2000, 0x3000, 0x4000)
    assert abi.STATUS[lib.gdn_kv_pages_grow(None, ctypes.byref(book), None, None, None, 1, 1, None,
                                            None, None, None)] == "GDN_ERR_ARG"
    assert abi.STATUS[lib.gdn_kv_pages_trim(None, ctypes.byref(book), None, None, 1, None)] == \
        "GDN_ERR_ARG"
    assert "kv" in lib.gdn_last_error_message().decode()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.fixture
def kv(monkeypatch):
    """A cache of 4 slots and 6 pages whose library calls all fail the test."""
    def launched(*_):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(
        gdn_kv_pages_grow=launched, gdn_kv_pages_trim=launched))
    return types.SimpleNamespace(handle=1, page_table=torch.full((4, 3), -1, dtype=torch.int32),
                                 desc=types.SimpleNamespace(n_slots=4, n_pages=6))


def refused(name, call, *args, **kw):
    with pytest.raises(abi.GDNError) as e:
        call(*args, **kw)
    assert e.value.name == name, e.value


def test_the_book_starts_with_every_page_free(kv):
    book = abi.KVPages(kv)
    assert book.held.tolist() == [0] * 4 and book.n_free.tolist() == [6]
    assert book.free_pages.tolist() == [5, 4, 3, 2, 1, 0]


def test_the_books_arrays_are_looked_at(kv):
    good = dict(held=i32(0, 0, 0, 0), free_pages=i32(*range(6)), n_free=i32(6))
    refused("GDN_ERR_ARG", abi.KVPages, kv, held=good["held"])
    refused("GDN_ERR_SIZE", abi.KVPages, kv, **{**good, "held": i32(0, 0)})
    refused("GDN_ERR_SIZE", abi.KVPages, kv, **{**good, "free_pages": i32(0)})
    refused("GDN_ERR_ARG", abi.KVPages, kv, **{**good, "n_free": i32(6).long()})
    refused("GDN_ERR_ARG", abi.KVPages, kv, **{**good, "held": i32(*range(8))[::2]})


def test_calls_with_wrong_arrays(kv):
    book = abi.KVPages(kv)
    grow, trim = abi.gdn_kv_pages_grow, abi.gdn_kv_pages_trim
    refused("GDN_ERR_ARG", grow, kv, book, i32(0).long(), i32(0), stream=STREAM)
    refused("GDN_ERR_SIZE", grow, kv, book, i32(0, 1), i32(0), stream=STREAM)
    refused("GDN_ERR_ARG", grow, kv, book, i32(0, 1), i32(0, 0), i32(0, 1, 2), stream=STREAM)
    refused("GDN_ERR_SIZE", grow, kv, book, i32(0, 1), i32(0, 0), i32(0, 1), 1, stream=STREAM)
    refused("GDN_ERR_SIZE", grow, kv, book, i32(0, 1), i32(0, 0), rows=torch.zeros(3).long(),
            stream=STREAM)
    refused("GDN_ERR_ARG", grow, kv, book, i32(0), i32(0), rows=i32(0), stream=STREAM)
    refused("GDN_ERR_ARG", grow, kv, book, i32(0), i32(0), positions=i32(0).long(), stream=STREAM)
    refused("GDN_ERR_SIZE", grow, kv, book, i32(0), i32(0), granted=i32(0, 0), stream=STREAM)
    refused("GDN_ERR_SIZE", grow, kv, book, i32(0), i32(0), None, 4, positions=i32(0),
            stream=STREAM)
    refused("GDN_ERR_ARG", grow, kv, book, torch.zeros(1, dtype=torch.int32, device="meta"),
            i32(0), stream=STREAM)
    refused("GDN_ERR_SIZE", trim, kv, book, i32(0, 1), i32(0), stream=STREAM)
    refused("GDN_ERR_ARG", trim, kv, book, i32(0, 1), i32(0, 0).long(), stream=STREAM)
