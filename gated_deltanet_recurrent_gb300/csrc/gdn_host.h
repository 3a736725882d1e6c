// Host helpers of the entry points: statuses with their messages, devices,
// index arrays brought to the host for the checks.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <vector>

#include "gdn_internal.h"

namespace gdn {
namespace host {

inline gdn_status fail(gdn_status s, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_message(buf);
  return s;
}

inline gdn_status ok() {
  set_last_message("");
  return GDN_OK;
}

inline gdn_status cuda_fail(cudaError_t e, const char *what) {
  return fail(GDN_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// The handle's device is the current one within the scope, whichever the caller has.
struct OnDevice {
  int before = -1;
  cudaError_t status;
  explicit OnDevice(int device) {
    status = cudaGetDevice(&before);
    if (status == cudaSuccess && before != device)
      status = cudaSetDevice(device);
    else
      before = -1;
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

inline bool dtype_ok(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }
inline size_t dtype_size(gdn_dtype d) { return d == GDN_F32 ? 4 : 2; }

inline gdn_status check_device_ptr(const void *ptr, const char *name) {
  cudaPointerAttributes attr;
  if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
    cudaGetLastError();
    return fail(GDN_ERR_ARG, "%s: cudaPointerGetAttributes failed", name);
  }
  if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
    return fail(GDN_ERR_ARG, "%s is not device memory", name);
  return GDN_OK;
}

inline gdn_status fetch(std::vector<int32_t> &dst, const int32_t *src, size_t n, cudaStream_t s,
                        const char *name) {
  dst.resize(n);
  if (n == 0) return GDN_OK;
  gdn_status st = check_device_ptr(src, name);
  if (st != GDN_OK) return st;
  cudaError_t e = cudaMemcpyAsync(dst.data(), src, n * sizeof(int32_t), cudaMemcpyDefault, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "copying index array to host");
  return GDN_OK;
}

}  // namespace host
}  // namespace gdn
