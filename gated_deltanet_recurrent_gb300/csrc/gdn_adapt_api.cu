// extern "C" entry points of the projection with adapters.
#include <new>
#include <vector>

#include "gdn_adapt.h"
#include "gdn_handles.h"
#include "gdn_host.h"

struct gdn_adapters {
  gdn_adapters_desc desc;
  const void *a, *b;
  const float *scale;
  int64_t ld_a, ld_b;
  int device;
  int sm_count;
  gdn::KVWork work;  // workspaces kept per stream, as the KV cache's
};

namespace {

using namespace gdn::host;

// Rows of bf16 elements whose starts are 16-byte aligned.  (A single row has no stride.)
gdn_status check_rows(const void *p, int64_t *ld, int64_t width, int64_t rows, const char *name) {
  if (rows == 1)
    *ld = (width + 7) / 8 * 8;
  else if (*ld == 0)
    *ld = width;
  if (*ld < width)
    return fail(GDN_ERR_ARG, "%s: row stride %lld smaller than a row of %lld", name,
                (long long)*ld, (long long)width);
  if ((uintptr_t)p % 16 || *ld % 8)
    return fail(GDN_ERR_ARG, "%s rows must start 16-byte aligned (pointer and stride)", name);
  return GDN_OK;
}

gdn_status check_ids(const gdn_adapters *ad, const int32_t *ids, int32_t tokens, cudaStream_t s) {
  try {
    std::vector<int32_t> h;
    gdn_status st = fetch(h, ids, (size_t)tokens, s, "ids");
    if (st != GDN_OK) return st;
    for (int32_t t = 0; t < tokens; ++t)
      if (h[t] < -1 || h[t] >= ad->desc.n_adapters)
        return fail(GDN_ERR_SIZE, "ids[%d] = %d outside [-1, %d)", t, h[t], ad->desc.n_adapters);
    return GDN_OK;
  } catch (const std::bad_alloc &) {
    return fail(GDN_ERR_SIZE, "no host memory to check the ids");
  }
}

}  // namespace

extern "C" {

gdn_status gdn_adapters_create(const gdn_adapters_desc *d, const void *a, int64_t ld_a,
                               const void *b, int64_t ld_b, const float *scale,
                               gdn_adapters **out) {
  if (!out) return fail(GDN_ERR_ARG, "out is NULL");
  *out = nullptr;
  if (!d) return fail(GDN_ERR_ARG, "desc is NULL");
  if (d->n_adapters < 1 || d->rank < 1 || d->hidden < 1 || d->n_out < 1)
    return fail(GDN_ERR_ARG, "adapter dimensions must be positive");
  if (d->rank > 128) return fail(GDN_ERR_UNSUPPORTED, "rank = %d (at most 128)", d->rank);
  // (k runs up to some thousands behind hidden)
  if (d->hidden > 1 << 30) return fail(GDN_ERR_UNSUPPORTED, "hidden = %d (at most 2^30)", d->hidden);
  // (rows of a and b are int32, and a tile's may lie up to 255 behind the last)
  if ((int64_t)d->n_adapters * d->n_out > INT32_MAX - 256 ||
      (int64_t)d->n_adapters * d->rank > INT32_MAX - 256)
    return fail(GDN_ERR_UNSUPPORTED, "n_adapters * n_out and * rank must stay below 2^31 - 256");
  if (!a || !b || !scale) return fail(GDN_ERR_ARG, "a, b and scale must be non-NULL");
  gdn_status st;
  if ((st = check_rows(a, &ld_a, d->hidden, (int64_t)d->n_adapters * d->rank, "a")) ||
      (st = check_rows(b, &ld_b, d->rank, (int64_t)d->n_adapters * d->n_out, "b")))
    return st;
  if ((uintptr_t)scale % 4) return fail(GDN_ERR_ARG, "scale must be 4-byte aligned");
  int dev = -1, sm_count = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (d->host_checks && ((st = check_device_ptr(a, "a")) || (st = check_device_ptr(b, "b")) ||
                         (st = check_device_ptr(scale, "scale"))))
    return st;
  e = cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(multiprocessor count)");
  gdn_adapters *ad = new (std::nothrow) gdn_adapters;
  if (!ad) return fail(GDN_ERR_SIZE, "no host memory for the handle");
  ad->desc = *d;
  ad->a = a, ad->b = b, ad->scale = scale, ad->ld_a = ld_a, ad->ld_b = ld_b;
  ad->device = dev, ad->sm_count = sm_count;
  ad->work.n = 0;
  cudaMemPoolProps props = {};
  props.allocType = cudaMemAllocationTypePinned;
  props.location.type = cudaMemLocationTypeDevice;
  props.location.id = dev;
  e = cudaMemPoolCreate(&ad->work.pool, &props);
  if (e == cudaSuccess) {
    uint64_t keep = UINT64_MAX;  // keep freed workspace for the next call
    e = cudaMemPoolSetAttribute(ad->work.pool, cudaMemPoolAttrReleaseThreshold, &keep);
    if (e != cudaSuccess) cudaMemPoolDestroy(ad->work.pool);
  }
  if (e != cudaSuccess) {
    delete ad;
    return cuda_fail(e, "creating the workspace memory pool");
  }
  *out = ad;
  return ok();
}

gdn_status gdn_adapters_destroy(gdn_adapters *ad) {
  if (!ad) return ok();
  const OnDevice here(ad->device);
  cudaError_t e = cudaDeviceSynchronize();
  if (here.status != cudaSuccess) e = here.status;
  cudaError_t e2 = cudaSuccess;
  for (int i = 0; i < ad->work.n; ++i) {
    const cudaError_t ew = cudaFree(ad->work.kept[i].mem);
    if (e2 == cudaSuccess) e2 = ew;
  }
  const cudaError_t e3 = cudaMemPoolDestroy(ad->work.pool);
  if (e2 == cudaSuccess) e2 = e3;
  delete ad;
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  if (e2 != cudaSuccess) return cuda_fail(e2, "releasing the adapters' handle");
  return ok();
}

gdn_status gdn_in_proj_adapted(gdn_pool *p, gdn_adapters *ad, int64_t tokens, const void *x,
                               int64_t ld_x, const void *w, int64_t ld_w, const int32_t *ids,
                               void *y, int64_t ld_y, gdn_dtype y_dtype, gdn_stream stream) {
  if (!p || !ad) return fail(GDN_ERR_ARG, "pool and adapters must be non-NULL");
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != p->device || dev != ad->device)
    return fail(GDN_ERR_ARG, "current device %d is not the pool's (%d) and the adapters' (%d)", dev,
                p->device, ad->device);
  if (tokens < 0) return fail(GDN_ERR_ARG, "tokens = %lld", (long long)tokens);
  if (!dtype_ok(y_dtype)) return fail(GDN_ERR_DTYPE, "y dtype must be F32 or BF16");
  if (tokens == 0) return ok();
  if (tokens > 1 << 18) return fail(GDN_ERR_SIZE, "tokens = %lld > 2^18", (long long)tokens);
  if (!x || !w || !ids || !y) return fail(GDN_ERR_ARG, "x, w, ids and y must be non-NULL");
  const gdn_adapters_desc &d = ad->desc;
  gdn_status st;
  if ((st = check_rows(x, &ld_x, d.hidden, tokens, "x")) ||
      (st = check_rows(w, &ld_w, d.hidden, d.n_out, "w")))
    return st;
  if (tokens == 1) ld_y = ((int64_t)d.n_out + 7) / 8 * 8;
  if (ld_y == 0) ld_y = d.n_out;
  if (ld_y < d.n_out) return fail(GDN_ERR_ARG, "y: row stride smaller than a row");
  if ((uintptr_t)y % 16 || (ld_y * (int64_t)dtype_size(y_dtype)) % 16)
    return fail(GDN_ERR_ARG, "y rows must start 16-byte aligned (pointer and stride)");
  if ((uintptr_t)ids % 4) return fail(GDN_ERR_ARG, "ids must be 4-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((p->desc.host_checks || d.host_checks) &&
      ((st = check_device_ptr(x, "x")) || (st = check_device_ptr(w, "w")) ||
       (st = check_device_ptr(y, "y")) || (st = check_ids(ad, ids, (int32_t)tokens, s))))
    return st;
  gdn::AdaptArgs g = {x, w, ad->a, ad->b, ad->scale, ids, y, ld_x, ld_w, ad->ld_a, ad->ld_b, ld_y,
                      (int)tokens, d.hidden, d.n_out, d.rank, d.n_adapters, y_dtype, nullptr, 0,
                      p->view.err, ad->sm_count, dev, p->view.test_flags};
  g.tile = gdn::adapt_tile(g);
  void *work = nullptr;
  bool temporary = false;
  e = ad->work.get(gdn::adapt_workspace_bytes(g), s, &work, &temporary);
  if (e != cudaSuccess) return cuda_fail(e, "the adapters' workspace");
  g.h = work;
  e = gdn::launch_adapt(g, s);
  if (temporary) {
    const cudaError_t ef = cudaFreeAsync(work, s);
    if (e == cudaSuccess) e = ef;
  }
  if (e == cudaErrorNotSupported)
    return fail(GDN_ERR_UNSUPPORTED, "no tensor map for these operands (driver entry point)");
  if (e != cudaSuccess) return cuda_fail(e, "adapted projection launch");
  return ok();
}

}  // extern "C"
