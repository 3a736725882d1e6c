"""gdn_kv_api.cu compiled as host code against a fake CUDA runtime, which keeps
a log of its calls and can be told to fail; the kernels' launchers are fakes
that keep their arguments.  (For what needs a second device or a failing call.)"""
import ctypes
import os
import subprocess

from gated_deltanet_recurrent_gb300 import abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_recurrent_gb300", "csrc")

FAKE = r"""
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <string>

#include "gdn_internal.h"

static int device = 0;
static std::string calls, message, failing;
static std::set<void *> live;
static gdn::KVAttendArgs attend_args;
static int rows_max_seqlen;

static cudaError_t call(const char *name) {
  calls += std::string(calls.empty() ? "" : " ") + name + "@" + std::to_string(device);
  return failing == name ? cudaErrorInvalidValue : cudaSuccess;
}
static cudaError_t alloc(const char *name, void **p, size_t n) {
  const cudaError_t e = call(name);
  if (e == cudaSuccess) live.insert(*p = malloc(n));
  return e;
}
static cudaError_t release(const char *name, void *p) {
  const cudaError_t e = call(name);
  if (e == cudaSuccess && p) {
    if (!live.erase(p)) abort();
    free(p);
  }
  return e;
}
static CUresult encode(CUtensorMap *, ...) { return CUDA_SUCCESS; }

extern "C" {
void fake_reset() { device = 0, calls = message = failing = ""; }
void fake_device(int d) { device = d; }
void fake_fail(const char *name) { failing = name; }
const char *fake_calls() { return calls.c_str(); }
int fake_live() { return (int)live.size(); }
int fake_max_seqlen() { return attend_args.max_seqlen; }
int fake_max_kv_len() { return attend_args.max_kv_len; }
int fake_rows_max_seqlen() { return rows_max_seqlen; }
const char *gdn_last_error_message() { return message.c_str(); }

cudaError_t cudaGetDevice(int *d) { return *d = device, cudaSuccess; }
cudaError_t cudaSetDevice(int d) { return device = d, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return call("synchronize"); }
cudaError_t cudaMalloc(void **p, size_t n) { return alloc("malloc", p, n); }
cudaError_t cudaFree(void *p) { return release("free", p); }
cudaError_t cudaMemset(void *p, int v, size_t n) { return memset(p, v, n), cudaSuccess; }
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, cudaMemcpyKind) {
  return memcpy(d, s, n), call("memcpy");
}
cudaError_t cudaMemcpyAsync(void *d, const void *s, size_t n, cudaMemcpyKind, cudaStream_t) {
  return memcpy(d, s, n), cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemPoolCreate(cudaMemPool_t *p, const cudaMemPoolProps *) {
  return alloc("pool_create", (void **)p, 8);
}
cudaError_t cudaMemPoolSetAttribute(cudaMemPool_t, cudaMemPoolAttr, void *) { return cudaSuccess; }
cudaError_t cudaMemPoolDestroy(cudaMemPool_t p) { return release("pool_destroy", p); }
cudaError_t cudaMallocFromPoolAsync(void **p, size_t n, cudaMemPool_t, cudaStream_t) {
  return alloc("pool_malloc", p, n);
}
cudaError_t cudaFreeAsync(void *p, cudaStream_t) { return release("free_async", p); }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus *s) {
  return *s = cudaStreamCaptureStatusNone, cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long *id) {
  return *id = (unsigned long long)(size_t)s, cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes *a, const void *) {
  return a->type = cudaMemoryTypeDevice, cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char *cudaGetErrorName(cudaError_t) { return "name"; }
const char *cudaGetErrorString(cudaError_t) { return "text"; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned int,
                                             unsigned long long, cudaDriverEntryPointQueryResult *q) {
  return *f = (void *)&encode, *q = cudaDriverEntryPointSuccess, cudaSuccess;
}

}  // extern "C"

static size_t workspace_bytes = 0;
extern "C" void fake_workspace_bytes(size_t n) { workspace_bytes = n; }

namespace gdn {
void set_last_message(const char *m) { message = m; }
cudaError_t launch_kv_append(const KVView &, int, const SeqIndex &, const int32_t *, int n,
                             const KVRows &, cudaStream_t) {
  return rows_max_seqlen = n, cudaSuccess;
}
cudaError_t launch_kv_read(const KVView &, int, const SeqIndex &, const int32_t *, int n,
                           const KVRows &, cudaStream_t) {
  return rows_max_seqlen = n, cudaSuccess;
}
cudaError_t launch_kv_attend(const KVView &, int, const KVAttendArgs &a, const KVHost &h,
                             cudaStream_t s) {
  attend_args = a;
  void *p;
  bool temporary;
  return workspace_bytes ? h.work->get(workspace_bytes, s, &p, &temporary) : cudaSuccess;
}
}  // namespace gdn
"""


def load(folder):
    src = os.path.join(str(folder), "fake.cc")
    out = os.path.join(str(folder), "libkvhost.so")
    with open(src, "w") as f:
        f.write(FAKE)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    # (-Bsymbolic: the fakes, not the runtime that the process may have loaded already)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-w", "-Wl,-Bsymbolic",
                    "-I", CSRC, "-I", cuda, "-x", "c++", src,
                    os.path.join(CSRC, "gdn_kv_api.cu"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    P = ctypes.POINTER
    for name, args in {
            "gdn_kv_create": [P(abi.gdn_kv_desc), vp, vp, ctypes.c_size_t, vp, vp, ctypes.c_size_t,
                              vp, P(vp)],
            "gdn_kv_destroy": [vp], "gdn_kv_get_error": [vp, P(ctypes.c_uint32)],
            "gdn_kv_append": [vp, i32, vp, vp, vp, i32, i32, i32, vp, i64, vp, i64, st, vp],
            "gdn_kv_read": [vp, i32, vp, vp, vp, i32, i32, i32, vp, i64, vp, i64, st, vp],
            "gdn_kv_attend": [vp, i32, vp, vp, vp, i32, i32, i32, i32, vp, i64, st, vp, i64, st,
                              ctypes.c_float, vp],
            "fake_fail": [ctypes.c_char_p], "fake_workspace_bytes": [ctypes.c_size_t]}.items():
        getattr(lib, name).argtypes = args
    lib.fake_calls.restype = lib.gdn_last_error_message.restype = ctypes.c_char_p
    return lib
