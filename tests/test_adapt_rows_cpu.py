"""A single row of x, w, y, a or b has no stride: whatever is given for one is not looked at, nor refused.  (The
entries' host code against a fake runtime, and the binding.)"""
import ctypes
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from tests.test_adapt_host_cpu import built, lib, run  # noqa: F401  (fixtures)


def create(lib, n=1, rank=1, hidden=100, n_out=1, ld_a=0, ld_b=0):
    out = ctypes.c_void_p()
    desc = abi.gdn_adapters_desc(n, rank, hidden, n_out, 0)
    st = lib.gdn_adapters_create(ctypes.byref(desc), 0x1000, ld_a, 0x2000, ld_b, 0x3000,
                                 ctypes.byref(out))
    return abi.STATUS[st], out


@pytest.mark.parametrize("ld", [0, 1, 100, 104, 3])
def test_single_rows(lib, ld):  # noqa: F811
    st, ad = create(lib, ld_a=ld, ld_b=ld)
    assert st == "GDN_OK"
    pool = lib.fake_pool(0)
    assert run(lib, pool, ad, tokens=1, ld_x=ld, ld_w=ld, ld_y=ld, dtype=abi.GDN_BF16) == "GDN_OK"
    assert [lib.fake_seen(i) for i in range(1, 6)] == [104, 104, 104, 8, 8]
    assert run(lib, pool, ad, tokens=1, x=0x4008) == "GDN_ERR_ARG"  # its start is
    assert run(lib, pool, ad, tokens=2, ld_x=100) == "GDN_ERR_ARG"
    assert run(lib, pool, ad, tokens=2, ld_x=104, ld_y=1) == "GDN_ERR_ARG"
    assert lib.gdn_adapters_destroy(ad) == 0


@pytest.mark.parametrize("kw", [dict(n=2, ld_a=100), dict(n=2, ld_a=104, ld_b=1), dict(rank=2),
                                dict(n_out=2), dict(n_out=2, ld_b=7)])
def test_several_rows_have_one(lib, kw):  # noqa: F811
    st, ad = create(lib, **kw)
    assert st == "GDN_ERR_ARG" and ad.value is None


def test_the_binding_lets_single_rows_through(monkeypatch):
    seen = []
    monkeypatch.setattr(abi, "gdn_adapters_create", lambda *a: seen.append(a))
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(
        gdn_in_proj_adapted=lambda *a: seen.append(a) or 0))
    bf = dict(dtype=torch.bfloat16)
    ad = abi.Adapters(torch.zeros(1, 1, 104, **bf)[..., :100], torch.zeros(1, 1, 1, **bf))
    ids, pool = torch.zeros(1, dtype=torch.int32), types.SimpleNamespace(handle=1)
    abi.gdn_in_proj_adapted(pool, ad, torch.zeros(1, 100, **bf), torch.zeros(1, 100, **bf), ids,
                            torch.zeros(1, 1, **bf), stream=types.SimpleNamespace(cuda_stream=0))
    assert len(seen) == 2
