"""The adapters' C entries on the host: devices, failing calls of the CUDA runtime, workspaces and
strides, against the fake runtime of tests/kv_host.py."""
import ctypes
import os
import subprocess

import pytest

from gated_deltanet_recurrent_gb300 import abi
from tests import kv_host

MORE = r"""
#include "gdn_adapt.h"
#include "gdn_handles.h"

static gdn::AdaptArgs seen;
static int launched;
extern "C" {
gdn_pool *fake_pool(int device) {
  gdn_pool *p = new gdn_pool();
  p->device = device;
  return p;
}
long long fake_seen(int what) {
  const long long v[] = {launched, seen.ld_x, seen.ld_w, seen.ld_a, seen.ld_b, seen.ld_y, seen.tokens,
                         seen.tile};
  return v[what];
}
cudaError_t fake_launch_result = cudaSuccess;
void fake_launch_fails(int e) { fake_launch_result = (cudaError_t)e; }
}
namespace gdn {
size_t adapt_workspace_bytes(const AdaptArgs &g) { return (size_t)g.tokens * 64; }
int adapt_tile(const AdaptArgs &g) { return g.tokens > 256 ? 256 : 0; }
cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t) {
  seen = g;
  ++launched;
  return fake_launch_result;
}
}  // namespace gdn
"""


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    folder = str(tmp_path_factory.mktemp("adapt_host"))
    src, out = os.path.join(folder, "fake.cc"), os.path.join(folder, "libadapthost.so")
    with open(src, "w") as f:
        f.write(kv_host.FAKE + MORE)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-w", "-Wl,-Bsymbolic", "-I",
                    kv_host.CSRC, "-I", cuda, "-x", "c++", src,
                    os.path.join(kv_host.CSRC, "gdn_kv_api.cu"),
                    os.path.join(kv_host.CSRC, "gdn_adapt_api.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    vp, i64, st, P = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.POINTER
    for name, args in {
            "gdn_adapters_create": [P(abi.gdn_adapters_desc), vp, i64, vp, i64, vp, P(vp)],
            "gdn_adapters_destroy": [vp],
            "gdn_in_proj_adapted": [vp, vp, i64, vp, i64, vp, i64, vp, vp, i64, st, vp],
            "fake_fail": [ctypes.c_char_p]}.items():
        getattr(lib, name).argtypes = args
    lib.fake_pool.restype = vp
    lib.fake_seen.restype = ctypes.c_longlong
    lib.fake_calls.restype = lib.gdn_last_error_message.restype = ctypes.c_char_p
    return lib


@pytest.fixture
def lib(built):
    built.fake_reset()
    built.fake_launch_fails(0)
    before = built.fake_live()
    yield built
    assert built.fake_live() == before, "something was not released"


def create(lib, rank=16, hidden=100, n_out=40, ld_a=104, ld_b=0):
    out = ctypes.c_void_p()
    desc = abi.gdn_adapters_desc(3, rank, hidden, n_out, 0)
    st = lib.gdn_adapters_create(ctypes.byref(desc), 0x1000, ld_a, 0x2000, ld_b, 0x3000,
                                 ctypes.byref(out))
    return st, out


def run(lib, pool, ad, tokens=5, x=0x4000, ld_x=104, w=0x5000, ld_w=104, ids=0x6000, y=0x7000,
        ld_y=0, dtype=abi.GDN_F32, stream=0):
    return abi.STATUS[lib.gdn_in_proj_adapted(pool, ad, tokens, x, ld_x, w, ld_w, ids, y, ld_y, dtype,
                                              stream)]


def test_arguments_that_launch_nothing(lib):
    _, ad = create(lib)
    pool = lib.fake_pool(0)
    before = lib.fake_seen(0)
    for kw, name in ((dict(tokens=-1), "GDN_ERR_ARG"), (dict(tokens=2 ** 18 + 1), "GDN_ERR_SIZE"),
                     (dict(dtype=abi.GDN_F16), "GDN_ERR_DTYPE"), (dict(x=None), "GDN_ERR_ARG"),
                     (dict(ids=None), "GDN_ERR_ARG"), (dict(y=None), "GDN_ERR_ARG"),
                     (dict(ld_x=96), "GDN_ERR_ARG"), (dict(ld_x=0), "GDN_ERR_ARG"),
                     (dict(ld_w=108), "GDN_ERR_ARG"), (dict(x=0x4008), "GDN_ERR_ARG"),
                     (dict(ld_y=39), "GDN_ERR_ARG"), (dict(ld_y=41), "GDN_ERR_ARG"),
                     (dict(y=0x7004), "GDN_ERR_ARG"), (dict(ids=0x6002), "GDN_ERR_ARG"),
                     (dict(dtype=abi.GDN_BF16, ld_y=44), "GDN_ERR_ARG"),
                     (dict(tokens=0, x=None, y=None, ids=None), "GDN_OK")):
        assert run(lib, pool, ad, **kw) == name, kw
    assert run(lib, None, ad) == run(lib, pool, None) == "GDN_ERR_ARG"
    assert lib.fake_seen(0) == before
    assert run(lib, pool, ad) == "GDN_OK"
    assert [lib.fake_seen(i) for i in range(1, 8)] == [104, 104, 104, 16, 40, 5, 0]
    assert lib.gdn_adapters_destroy(ad) == 0


def test_another_device_is_refused_and_a_handle_released_on_its_own(lib):
    _, ad = create(lib)
    assert run(lib, lib.fake_pool(3), ad) == "GDN_ERR_ARG"
    assert run(lib, lib.fake_pool(0), ad) == "GDN_OK"
    lib.fake_device(3)
    assert run(lib, lib.fake_pool(0), ad) == "GDN_ERR_ARG"
    assert run(lib, lib.fake_pool(3), ad) == "GDN_ERR_ARG"
    lib.fake_reset()
    lib.fake_device(3)
    assert lib.gdn_adapters_destroy(ad) == 0
    calls = lib.fake_calls().decode().split()
    assert calls[0] == "synchronize@0" and all(c.endswith("@0") for c in calls), calls


@pytest.mark.parametrize("call", ["pool_create"])
def test_a_handle_that_cannot_be_made_leaves_nothing(lib, call):
    lib.fake_fail(call.encode())
    st, out = create(lib)
    assert abi.STATUS[st] == "GDN_ERR_CUDA" and out.value is None


def test_workspaces_are_kept_per_stream_and_grow(lib):
    _, ad = create(lib)
    pool = lib.fake_pool(0)
    lib.fake_reset()
    for stream, tokens in ((1, 5), (1, 5), (2, 5), (1, 3), (1, 500), (1, 500)):
        assert run(lib, pool, ad, tokens=tokens, stream=stream) == "GDN_OK"
    calls = [c.split("@")[0] for c in lib.fake_calls().decode().split()]
    assert calls == ["pool_malloc", "pool_malloc", "free_async", "pool_malloc"]
    assert lib.fake_seen(7) == 256
    assert lib.gdn_adapters_destroy(ad) == 0


def test_failures_leave_the_handle_usable(lib):
    _, ad = create(lib)
    pool = lib.fake_pool(0)
    lib.fake_fail(b"pool_malloc")
    assert run(lib, pool, ad) == "GDN_ERR_CUDA"
    lib.fake_fail(b"")
    lib.fake_launch_fails(801)  # cudaErrorNotSupported: no tensor map
    assert run(lib, pool, ad) == "GDN_ERR_UNSUPPORTED"
    lib.fake_launch_fails(1)
    assert run(lib, pool, ad) == "GDN_ERR_CUDA"
    lib.fake_launch_fails(0)
    assert run(lib, pool, ad) == "GDN_OK"
    assert lib.gdn_adapters_destroy(ad) == 0
