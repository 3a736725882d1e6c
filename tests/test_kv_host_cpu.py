"""The KV cache's C entries on the host: devices, failing calls of the CUDA
runtime and the bounds that reach the launchers, against a fake runtime."""
import ctypes

import pytest

from gated_deltanet_recurrent_gb300 import abi
from tests import kv_host


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    return kv_host.load(tmp_path_factory.mktemp("kv_host"))


@pytest.fixture
def lib(built):
    built.fake_reset()
    built.fake_workspace_bytes(0)
    before = built.fake_live()
    yield built
    assert built.fake_live() == before, "something was not released"


def create(lib, **kw):
    d = dict(n_layers=1, n_slots=4, n_pages=8, max_pages=2, page_tokens=16, h_q=8, h_kv=2, d=64,
             code=abi.GDN_KV_I8, host_checks=0)
    d.update(kw)
    out = ctypes.c_void_p()
    st = lib.gdn_kv_create(ctypes.byref(abi.gdn_kv_desc(**d)), 0x1000, 0x2000, 1 << 50, 0x3000,
                           0x4000, 1 << 50, 0x5000, ctypes.byref(out))
    assert st == 0, lib.gdn_last_error_message()
    return out


def attend(lib, kv, cu=None, n_seqs=1, tokens=1, max_seqlen=1, max_kv_len=1, stream=0):
    return lib.gdn_kv_attend(kv, 0, 0x6000, 0x7000, cu, n_seqs, tokens, max_seqlen, max_kv_len,
                             0x8000, 0, abi.GDN_BF16, 0x9000, 0, abi.GDN_BF16, 1.0, stream)


def test_a_handle_is_released_on_its_own_device(lib):
    """(A garbage collector may run the destructor with any device current.)"""
    kv = create(lib)
    lib.fake_workspace_bytes(100)
    assert attend(lib, kv) == 0
    lib.fake_reset()
    lib.fake_device(3)
    assert lib.gdn_kv_destroy(kv) == 0
    calls = lib.fake_calls().decode().split()
    assert calls[0] == "synchronize@0" and all(c.endswith("@0") for c in calls), calls
    device = ctypes.c_int(-1)
    lib.cudaGetDevice(ctypes.byref(device))
    assert device.value == 3


def test_the_error_word_is_read_on_its_own_device(lib):
    kv = create(lib)
    lib.fake_reset()
    lib.fake_device(2)
    err = ctypes.c_uint32(7)
    assert lib.gdn_kv_get_error(kv, ctypes.byref(err)) == 0 and err.value == 0
    calls = lib.fake_calls().decode().split()
    assert calls and all(c.endswith("@0") for c in calls), calls
    device = ctypes.c_int(-1)
    lib.cudaGetDevice(ctypes.byref(device))
    assert device.value == 2
    assert lib.gdn_kv_destroy(kv) == 0


def test_a_workspace_that_grows_loses_no_memory_when_a_call_fails(lib):
    kv = create(lib)
    lib.fake_workspace_bytes(100)
    assert attend(lib, kv, stream=1) == 0
    lib.fake_workspace_bytes(200)
    for name in (b"free_async", b"pool_malloc"):
        lib.fake_fail(name)
        assert abi.STATUS[attend(lib, kv, stream=1)] == "GDN_ERR_CUDA"
    lib.fake_fail(b"")
    before = lib.fake_live()
    assert attend(lib, kv, stream=1) == 0
    assert lib.fake_live() == before + 1     # (the failed growth had given the old one back)
    lib.fake_reset()
    for n in (200, 150, 10):                 # what is there serves smaller calls
        lib.fake_workspace_bytes(n)
        assert attend(lib, kv, stream=1) == 0
    assert lib.fake_calls() == b""
    assert lib.gdn_kv_destroy(kv) == 0


HUGE = 2 ** 31 - 1


def test_loose_bounds_are_cut_to_what_a_call_can_hold(lib):
    """A caller that captures a graph gives a loose bound: it must not size a
    grid of two thousand million CTAs for a handful of tokens."""
    kv = create(lib)
    rows = (0x8000, 0, 0x9000, 0, abi.GDN_BF16, None)
    for hint, want in ((HUGE, 50), (50, 50), (20, 20), (1, 1), (0, 1), (-5, 1)):
        assert attend(lib, kv, cu=0xa000, n_seqs=3, tokens=50, max_seqlen=hint) == 0
        assert lib.fake_max_seqlen() == want
        for call in (lib.gdn_kv_append, lib.gdn_kv_read):
            assert call(kv, 0, 0x6000, 0x7000, 0xa000, 3, 50, hint, *rows) == 0
            assert lib.fake_rows_max_seqlen() == want
    # one token each: no sequence is longer
    assert attend(lib, kv, n_seqs=3, tokens=3, max_seqlen=HUGE) == 0
    assert lib.fake_max_seqlen() == 1
    assert lib.gdn_kv_append(kv, 0, 0x6000, 0x7000, None, 3, 3, HUGE, *rows) == 0
    assert lib.fake_rows_max_seqlen() == 1
    # a slot holds 2 pages of 16
    for hint, want in ((HUGE, 32), (32, 32), (7, 7), (0, 1)):
        assert attend(lib, kv, max_kv_len=hint) == 0
        assert lib.fake_max_kv_len() == want
    assert lib.gdn_kv_destroy(kv) == 0
