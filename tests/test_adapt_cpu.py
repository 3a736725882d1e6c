"""What the projection with adapters refuses before any launch."""
import ctypes
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from gated_deltanet_recurrent_gb300 import build as gbuild


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return abi.load_library()


@pytest.mark.parametrize("kw,name", [
    (dict(n_adapters=0), "GDN_ERR_ARG"), (dict(rank=0), "GDN_ERR_ARG"),
    (dict(hidden=0), "GDN_ERR_ARG"), (dict(n_out=-3), "GDN_ERR_ARG"),
    (dict(rank=129), "GDN_ERR_UNSUPPORTED"), (dict(n_adapters=2 ** 24), "GDN_ERR_UNSUPPORTED"),
    (dict(a=None), "GDN_ERR_ARG"), (dict(b=None), "GDN_ERR_ARG"), (dict(scale=None), "GDN_ERR_ARG"),
    (dict(ld_a=63), "GDN_ERR_ARG"), (dict(ld_b=4), "GDN_ERR_ARG"), (dict(ld_a=68), "GDN_ERR_ARG"),
    (dict(rank=12), "GDN_ERR_ARG"), (dict(b=0x2008), "GDN_ERR_ARG"),
    (dict(scale=0x3002), "GDN_ERR_ARG")])
def test_handles_that_cannot_be(lib, kw, name):
    v = dict(n_adapters=4, rank=8, hidden=64, n_out=256, a=0x1000, ld_a=0, b=0x2000, ld_b=0,
             scale=0x3000)
    v.update(kw)
    desc = abi.gdn_adapters_desc(v["n_adapters"], v["rank"], v["hidden"], v["n_out"], 0)
    out = ctypes.c_void_p()
    st = lib.gdn_adapters_create(ctypes.byref(desc), v["a"], v["ld_a"], v["b"], v["ld_b"],
                                 v["scale"], ctypes.byref(out))
    assert abi.STATUS[st] == name and out.value is None


def test_null_handles_fail_cleanly(lib):
    st = lib.gdn_in_proj_adapted(None, None, 1, None, 0, None, 0, None, None, 0, 0, None)
    assert abi.STATUS[st] == "GDN_ERR_ARG"
    assert lib.gdn_adapters_destroy(None) == 0
    assert abi.STATUS[lib.gdn_adapters_create(None, None, 0, None, 0, None,
                                              ctypes.byref(ctypes.c_void_p()))] == "GDN_ERR_ARG"


@pytest.fixture
def made(monkeypatch):
    """Descriptors and strides that reach gdn_adapters_create, which makes nothing."""
    seen = []
    monkeypatch.setattr(abi, "gdn_adapters_create",
                        lambda desc, a, ld_a, b, ld_b, scale: seen.append((desc, ld_a, ld_b)))
    return seen


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_strides_of_the_adapters(made):
    abi.Adapters(z(3, 8, 64), z(3, 32, 8))
    abi.Adapters(z(3, 8, 80)[..., :64], z(3, 32, 16)[..., :8])
    abi.Adapters(z(1, 1, 64), z(1, 1, 1))
    assert [(a, b) for _, a, b in made] == [(64, 8), (80, 16), (64, 1)]


@pytest.mark.parametrize("a,b,scale,name", [
    (z(3, 8, 64, dtype=torch.float32), z(3, 32, 8), None, "GDN_ERR_DTYPE"),
    (z(3, 8, 64), z(2, 32, 8), None, "GDN_ERR_SIZE"),
    (z(3, 8, 64), z(3, 32, 16), None, "GDN_ERR_SIZE"),
    (z(3, 64), z(3, 32, 8), None, "GDN_ERR_SIZE"),
    (z(3, 8, 64), z(3, 32, 8), z(2, dtype=torch.float32), "GDN_ERR_ARG"),
    (z(3, 8, 64), z(3, 32, 8), z(3), "GDN_ERR_ARG"),
    (z(3, 16, 64)[:, ::2], z(3, 32, 8)[:, :, :], None, None),
    (z(6, 8, 64)[::2], z(3, 32, 8), None, "GDN_ERR_ARG"),
    (z(3, 8, 1).expand(3, 8, 64), z(3, 32, 8), None, "GDN_ERR_ARG"),
    (z(1, 8, 64).expand(3, 8, 64), z(3, 32, 8), None, "GDN_ERR_ARG"),
    (z(3, 64, 8).transpose(1, 2), z(3, 32, 8), None, "GDN_ERR_ARG"),
    (z(3, 8, 64), z(3, 8, 32).transpose(1, 2), None, "GDN_ERR_ARG")])
def test_adapters_the_binding_refuses(made, a, b, scale, name):
    if name is None:
        abi.Adapters(a, b, scale)
        return
    with pytest.raises(abi.GDNError) as e:
        abi.Adapters(a, b, scale)
    assert e.value.name == name


def test_calls_the_binding_refuses(made, monkeypatch):
    def launched(*_):
        raise AssertionError("the call reached the library")
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(gdn_in_proj_adapted=launched))
    ad = abi.Adapters(z(3, 8, 64), z(3, 32, 8))
    pool = types.SimpleNamespace(handle=1)
    ids = torch.zeros(5, dtype=torch.int32)
    x, w, y = z(5, 64), z(32, 64), z(5, 32)

    def refused(name, *args):
        with pytest.raises(abi.GDNError) as e:
            abi.gdn_in_proj_adapted(pool, ad, *args, stream=types.SimpleNamespace(cuda_stream=0))
        assert e.value.name == name, e.value
    refused("GDN_ERR_DTYPE", x.float(), w, ids, y)
    refused("GDN_ERR_DTYPE", x, w.half(), ids, y)
    refused("GDN_ERR_DTYPE", x, w, ids, y.double())
    refused("GDN_ERR_ARG", x, w, ids.long(), y)
    refused("GDN_ERR_ARG", x, w, torch.zeros(10, dtype=torch.int32)[::2], y)
    refused("GDN_ERR_SIZE", x[:4], w, ids, y)
    refused("GDN_ERR_SIZE", x, w[:31], ids, y)
    refused("GDN_ERR_SIZE", x, w, ids, y[:, :31])
    refused("GDN_ERR_ARG", x[:1].expand(5, 64), w, ids, y)
    refused("GDN_ERR_ARG", x, w, ids, y[:1].expand(5, 32))
    refused("GDN_ERR_ARG", x, z(64, 32).T, ids, y)
    refused("GDN_ERR_ARG", torch.zeros(5, 64, dtype=torch.bfloat16, device="meta"), w, ids, y)


@pytest.mark.parametrize("cls,call", [
    (abi.Adapters, "gdn_adapters_destroy"), (abi.Rope, "gdn_rope_destroy"),
    (abi.Pool, "gdn_pool_destroy"), (abi.KVCache, "gdn_kv_destroy")])
def test_a_destroy_call_that_reports_an_error_is_not_made_again(monkeypatch, cls, call):
    """The library frees a handle even where the device has failed."""
    freed = []

    def destroy(handle):
        freed.append(handle)
        return 7 if handle else 0

    fake = types.SimpleNamespace(**{call: destroy, "gdn_last_error_message": lambda: b"no device"})
    monkeypatch.setattr(abi, "load_library", lambda: fake)
    owner = cls.__new__(cls)
    owner.handle = 1234
    with pytest.raises(abi.GDNError):
        owner.close()
    owner.close()
    owner.__del__()
    assert freed == [1234]
    owner.handle = 5678  # by the function itself
    with pytest.raises(abi.GDNError):
        getattr(abi, call)(owner)
    owner.__del__()
    assert freed == [1234, 5678]
