"""held and free_pages belong to one cache: with another on the same page table, of more slots or pages, the kernels
would run past their ends."""
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

STREAM = types.SimpleNamespace(cuda_stream=0)


def cache(table, n_slots, n_pages):
    return types.SimpleNamespace(handle=1, page_table=table,
                                 desc=types.SimpleNamespace(n_slots=n_slots, n_pages=n_pages))


@pytest.mark.parametrize("n_slots,n_pages", [(4, 7), (4, 5), (5, 6), (3, 6)])
def test_a_book_of_another_cache(monkeypatch, n_slots, n_pages):
    calls = []
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(
        gdn_kv_pages_grow=lambda *a: calls.append(a) or 0,
        gdn_kv_pages_trim=lambda *a: calls.append(a) or 0))
    table = torch.full((4, 3), -1, dtype=torch.int32)
    own, other = cache(table, 4, 6), cache(table, n_slots, n_pages)
    book = abi.KVPages(own)
    ids = torch.tensor([2, 0], dtype=torch.int32)
    for call in (abi.gdn_kv_pages_grow, abi.gdn_kv_pages_trim):
        with pytest.raises(abi.GDNError) as e:
            call(other, book, ids, torch.zeros_like(ids), stream=STREAM)
        assert e.value.name == "GDN_ERR_SIZE" and not calls
    for call in (abi.gdn_kv_pages_grow, abi.gdn_kv_pages_trim):
        call(own, book, ids, torch.zeros_like(ids), stream=STREAM)
    assert len(calls) == 2
