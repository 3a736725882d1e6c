"""Row strides that the Python binding refuses before any launch: the library
reads a stride of 0 as "packed", so rows expanded from one would be read, or
written, past the one row."""
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

POOL = types.SimpleNamespace(handle=1, desc=types.SimpleNamespace(h_k=2, dk=16, h_v=2, dv=8))
STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def launched(*_):
        raise AssertionError("the call reached the library")
    names = ("gdn_conv_silu", "gdn_decode_step", "gdn_decode_step_conv", "gdn_in_proj",
             "gdn_prefill_chunked")
    fake = types.SimpleNamespace(**{n: launched for n in names})
    monkeypatch.setattr(abi, "load_library", lambda: fake)


def refused(call, *args, **kw):
    with pytest.raises(abi.GDNError) as e:
        call(POOL, *args, stream=STREAM, **kw)
    assert e.value.name == "GDN_ERR_ARG" and "stride" in str(e.value)


def one(*shape):
    """A tensor of `shape` whose rows are all the same memory."""
    return torch.zeros(1, *shape[1:]).expand(*shape)


def test_expanded_tokens_are_refused():
    n = 5
    ids = torch.zeros(n, dtype=torch.int32)
    q, v, g, o = (torch.zeros(n, 2, 16), torch.zeros(n, 2, 8), torch.zeros(n, 2),
                  torch.zeros(n, 2, 8))
    refused(abi.gdn_decode_step, 0, ids, one(n, 2, 16), one(n, 2, 16), v, g, g, o)
    refused(abi.gdn_decode_step, 0, ids, q, q, one(n, 2, 8), g, g, o)
    cu = torch.zeros(n + 1, dtype=torch.int32)
    refused(abi.gdn_prefill_chunked, 0, ids, cu, q, q, one(n, 2, 8), g, g, o)


def test_expanded_rows_are_refused():
    n, c = 5, 80
    ids = torch.zeros(n, dtype=torch.int32)
    w, x, g = torch.zeros(c, 4), torch.zeros(n, c), torch.zeros(n, 2)
    refused(abi.gdn_conv_silu, 0, ids, one(n, c), w, x)
    refused(abi.gdn_conv_silu, 0, ids, x, w, one(n, c))
    o = torch.zeros(n, 2, 8)
    refused(abi.gdn_decode_step_conv, 0, ids, one(n, c), w, x, g, g, o)
    refused(abi.gdn_decode_step_conv, 0, ids, x, w, one(n, c), g, g, o)
    a, b, y = torch.zeros(4, 32).bfloat16(), torch.zeros(8, 32).bfloat16(), torch.zeros(4, 8)
    refused(abi.gdn_in_proj, one(4, 32).bfloat16(), b, one(4, 8))
    refused(abi.gdn_in_proj, a[:1].expand(4, 32), b, y)
    refused(abi.gdn_in_proj, a, b[:1].expand(8, 32), y)


def test_a_single_row_keeps_its_width():
    """(not 0: a row narrower than the layer's channels has to be refused by the library)"""
    assert abi._row_stride(one(1, 7), 7, "x") == 7
    assert abi._row_stride(torch.zeros(3, 9)[:, :7], 7, "x") == 9
    assert abi._token_rows(torch.zeros(1, 2, 16).expand(1, 2, 16), 2, 16, "q") == 32
