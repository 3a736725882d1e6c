"""What the Python binding of the 8-bit KV cache refuses before any launch."""
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi

STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture
def kv(monkeypatch):
    """A cache of 2 KV heads of 64 whose library calls all fail the test."""
    def launched(*_):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(
        gdn_kv_append=launched, gdn_kv_read=launched, gdn_kv_attend=launched))
    return types.SimpleNamespace(handle=1, h_q=4, h_kv=2, d=64,
                                 desc=types.SimpleNamespace(max_pages=4, page_tokens=16))


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def refused(call, *args, **kw):
    with pytest.raises(abi.GDNError) as e:
        call(*args, stream=STREAM, **kw)
    assert e.value.name == "GDN_ERR_ARG" and "stride" in str(e.value)


def test_expanded_rows_are_refused(kv):
    """One row broadcast over several tokens has the stride 0, which the C
    calls take for packed rows: they would read past the one row."""
    good, row = torch.zeros(9, 2, 64), torch.zeros(1, 2, 64).expand(9, 2, 64)
    args = (kv, 0, i32(1), i32(0))
    cu = i32(0, 9)
    for k, v in ((row, good), (good, row)):
        refused(abi.gdn_kv_append, *args, k, v, cu_seqlens=cu)
        refused(abi.gdn_kv_read, *args, k, v, cu_seqlens=cu)
    refused(abi.gdn_kv_read, *args, row, None, cu_seqlens=cu)
    q, q_row = torch.zeros(9, 4, 64), torch.zeros(1, 4, 64).expand(9, 4, 64)
    refused(abi.gdn_kv_attend, *args, q_row, q, cu_seqlens=cu)
    refused(abi.gdn_kv_attend, *args, q, q_row, cu_seqlens=cu)


def test_overlapping_rows_are_refused(kv):
    over = torch.zeros(2000).as_strided((9, 2, 64), (64, 64, 1))
    refused(abi.gdn_kv_append, kv, 0, i32(1), i32(0), over, over, cu_seqlens=i32(0, 9))


def test_the_stride_of_a_single_row_says_nothing():
    row = torch.zeros(1, 2, 64).expand(1, 2, 64)
    assert abi._kv_token_rows(row.shape, (0, 64, 1), 2, 64, "k") == 0
    assert abi._kv_token_rows((0, 2, 64), (128, 64, 1), 2, 64, "k") == 0
    assert abi._kv_token_rows((3, 2, 64), (384, 64, 1), 2, 64, "k") == 384


def test_the_stride_of_a_single_head_says_nothing():
    x = torch.zeros(5, 3, 64)[:, 1:2]                # packed rows' second head: strides 192, 64
    assert abi._kv_token_rows(x.shape, x.stride(), 1, 64, "k") == 192
    x = torch.zeros(1, 5, 64).transpose(0, 1)        # [5, 1, 64] of strides 64, 320
    assert x.stride(1) == 320
    assert abi._kv_token_rows(x.shape, x.stride(), 1, 64, "k") == 64
    assert abi._token_rows(x, 1, 64, "q") == 64
    with pytest.raises(abi.GDNError):
        abi._kv_token_rows((5, 2, 64), (640, 320, 1), 2, 64, "k")


def test_unknown_test_flags_fail_cleanly():
    from gated_deltanet_recurrent_gb300 import build
    build.build()
    lib = abi.load_library()
    assert abi.STATUS[lib.gdn_kv_set_test_flags(None, 1)] == "GDN_ERR_ARG"
