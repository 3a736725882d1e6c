"""What gdn_rope refuses before any launch, at the C entries and in the binding."""
import ctypes
import math
import types

import pytest
import torch

from gated_deltanet_recurrent_gb300 import abi
from gated_deltanet_recurrent_gb300 import build as gbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return abi.load_library()


@pytest.mark.parametrize("kw,name", [
    (dict(d=63), "GDN_ERR_ARG"), (dict(rot=0), "GDN_ERR_ARG"), (dict(rot=7), "GDN_ERR_ARG"),
    (dict(rot=66), "GDN_ERR_ARG"), (dict(d=1024, rot=514), "GDN_ERR_UNSUPPORTED"),
    (dict(d=4098), "GDN_ERR_UNSUPPORTED"), (dict(layout="quarter"), "GDN_ERR_ARG"),
    (dict(base=0.0), "GDN_ERR_ARG"), (dict(base=math.inf), "GDN_ERR_ARG"),
    (dict(base=math.nan), "GDN_ERR_ARG"), (dict(factor=0.0), "GDN_ERR_ARG"),
    (dict(factor=-2.0), "GDN_ERR_ARG"), (dict(original_len=-1), "GDN_ERR_ARG"),
    (dict(original_len=8, low_turns=4.0, high_turns=4.0), "GDN_ERR_ARG"),
    (dict(original_len=8, low_turns=-1.0), "GDN_ERR_ARG"),
    (dict(original_len=8, high_turns=math.inf), "GDN_ERR_ARG"),
    (dict(out_scale=math.nan), "GDN_ERR_ARG")])
def test_plans_that_cannot_be(kw, name):
    with pytest.raises(abi.GDNError) as e:
        abi.Rope(**{"d": 64, "rot": 64, **kw})
    assert e.value.name == name


@pytest.mark.parametrize("kw", [
    dict(base=1e-320), dict(factor=1e-320), dict(base=1e-300, factor=1e-300),
    dict(base=1e-300, factor=1e-300, original_len=8, low_turns=0.5, high_turns=1e308)])
def test_frequencies_that_are_not_finite(kw):
    with pytest.raises(abi.GDNError) as e:
        abi.Rope(**{"d": 64, "rot": 64, **kw})
    assert e.value.name == "GDN_ERR_ARG"


def test_a_plan_needs_no_device():
    rope = abi.Rope(256, 64)
    rope.close()
    rope.close()


def call(lib, plan, tokens=3, positions=0x1000, q=0x2000, ld_q=0, h_q=2, k=0x4000, ld_k=0, h_k=1,
         q_out=0x6000, ld_q_out=0, k_out=0x8000, ld_k_out=0, dtype=abi.GDN_BF16):
    return abi.STATUS[lib.gdn_rope(plan, tokens, positions, q, ld_q, h_q, k, ld_k, h_k, q_out,
                                   ld_q_out, k_out, ld_k_out, dtype, None)]


def test_calls_that_launch_nothing(lib):
    rope = abi.Rope(64)
    p = rope.handle
    assert call(lib, None) == "GDN_ERR_ARG"
    assert call(lib, p, tokens=-1) == call(lib, p, h_q=-1) == "GDN_ERR_ARG"
    assert call(lib, p, positions=None) == call(lib, p, q=None) == "GDN_ERR_ARG"
    assert call(lib, p, k_out=None) == "GDN_ERR_ARG"
    assert call(lib, p, dtype=abi.GDN_F16) == call(lib, p, dtype=9) == "GDN_ERR_DTYPE"
    assert call(lib, p, ld_q=127) == call(lib, p, ld_k_out=63) == "GDN_ERR_ARG"
    assert call(lib, p, q=0x2001) == "GDN_ERR_ARG"
    assert call(lib, p, dtype=abi.GDN_F32, k=0x4002) == "GDN_ERR_ARG"
    assert call(lib, p, q_out=0x2000, ld_q=256, ld_q_out=128) == "GDN_ERR_ARG"
    assert call(lib, p, h_k=70000) == "GDN_ERR_UNSUPPORTED"
    assert call(lib, p, tokens=0, positions=None, q=None) == "GDN_OK"
    assert call(lib, p, h_q=0, h_k=0, q=None, k=None) == "GDN_OK"
    assert lib.gdn_rope_create(None, ctypes.byref(ctypes.c_void_p())) == 1
    assert lib.gdn_rope_create(ctypes.byref(rope.desc), None) == 1
    assert lib.gdn_rope_destroy(None) == 0


def test_the_binding_refuses(monkeypatch):
    """Tensors that say `cuda` where they are looked at, and a library that must not be reached."""
    rope = abi.Rope(64)

    def launched(*_):
        raise AssertionError("the call reached the library")
    real = abi._lib
    monkeypatch.setattr(abi, "_lib", types.SimpleNamespace(
        gdn_rope=launched, gdn_rope_destroy=real.gdn_rope_destroy))

    def refused(name, *args, **kw):
        with pytest.raises(abi.GDNError) as e:
            abi.gdn_rope(rope, *args, stream=types.SimpleNamespace(cuda_stream=0), **kw)
        assert e.value.name == name, e.value
    at = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 2, 64)
    refused("GDN_ERR_ARG", at, None)
    refused("GDN_ERR_ARG", at, q)          # a CPU tensor
    refused("GDN_ERR_DTYPE", at, q.half())
    rows = lambda x, out=None, n=3: abi._rope_rows(x, out, 64, n, torch.float32, at.get_device(), "q")
    for x, out in ((q[:2], None), (q[..., :32], None), (q, q[:, :1]), (q[:, 0], None)):
        with pytest.raises(abi.GDNError) as e:
            rows(x, out)
        assert e.value.name == "GDN_ERR_SIZE"
    for x, out in ((q.transpose(0, 1).contiguous().transpose(0, 1), None),
                   (q[:1].expand(3, 2, 64), None), (q, q[:1].expand(3, 2, 64))):
        with pytest.raises(abi.GDNError) as e:
            rows(x, out)
        assert e.value.name == "GDN_ERR_ARG"
    with pytest.raises(abi.GDNError) as e:
        rows(q, q.double())
    assert e.value.name == "GDN_ERR_DTYPE"
    monkeypatch.undo()
