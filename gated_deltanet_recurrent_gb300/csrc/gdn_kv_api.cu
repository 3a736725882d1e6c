// extern "C" entry points of the 8-bit paged KV cache: argument validation
// (always), optional host-side validation of the index arrays and of the page
// table entries in use, and the kernel launches.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <new>
#include <vector>

#include "gdn_handles.h"
#include "gdn_host.h"

namespace gdn {

cudaError_t KVWork::get(size_t bytes, cudaStream_t s, void **mem, bool *temporary) {
  *temporary = true;
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  cudaError_t e = cudaStreamIsCapturing(s, &capture);
  if (e != cudaSuccess) return e;
  if (capture == cudaStreamCaptureStatusNone) {
    if ((e = cudaStreamGetId(s, &id)) != cudaSuccess) return e;
    int i = 0;
    while (i < n && kept[i].stream != id) ++i;
    if (i < n && kept[i].bytes >= bytes) {
      *temporary = false;
      *mem = kept[i].mem;
      return cudaSuccess;
    }
    if (i < kStreams) {  // a new stream, or a larger call than before
      // (a call that fails leaves the place as it is, or empty: nothing is lost)
      if (i < n && kept[i].mem) {
        e = cudaFreeAsync(kept[i].mem, s);
        if (e != cudaSuccess) return e;
      }
      kept[i] = {id, nullptr, 0};
      if (i == n) ++n;
      e = cudaMallocFromPoolAsync(&kept[i].mem, bytes, pool, s);
      if (e != cudaSuccess) {
        kept[i].mem = nullptr;
        return e;
      }
      kept[i].bytes = bytes;
      *temporary = false;
      *mem = kept[i].mem;
      return cudaSuccess;
    }
  }
  return cudaMallocFromPoolAsync(mem, bytes, pool, s);
}

}  // namespace gdn

namespace {

using namespace gdn::host;

gdn_status check_desc(const gdn_kv_desc *d) {
  if (!d) return fail(GDN_ERR_ARG, "desc is NULL");
  if (d->n_layers < 1 || d->n_slots < 1 || d->n_pages < 1 || d->max_pages < 1 || d->h_q < 1 ||
      d->h_kv < 1)
    return fail(GDN_ERR_ARG, "cache dimensions must be positive");
  if (d->h_q % d->h_kv != 0)
    return fail(GDN_ERR_ARG, "h_q (%d) is not a multiple of h_kv (%d)", d->h_q, d->h_kv);
  if (d->code != GDN_KV_I8 && d->code != GDN_KV_E4M3)
    return fail(GDN_ERR_DTYPE, "code must be GDN_KV_I8 or GDN_KV_E4M3");
  if (d->d != 64 && d->d != 128 && d->d != 256)
    return fail(GDN_ERR_UNSUPPORTED, "d=%d (supported: 64, 128, 256)", d->d);
  if (d->page_tokens != 16 && d->page_tokens != 32 && d->page_tokens != 64 &&
      d->page_tokens != 128)
    return fail(GDN_ERR_UNSUPPORTED, "page_tokens=%d (supported: 16, 32, 64, 128)",
                d->page_tokens);
  if (d->n_slots > 65535) return fail(GDN_ERR_UNSUPPORTED, "n_slots=%d (max 65535)", d->n_slots);
  if (d->h_kv > 4096 || d->h_q / d->h_kv > 4096)
    return fail(GDN_ERR_UNSUPPORTED, "more than 4096 KV heads or query heads per KV head");
  if ((int64_t)d->n_layers * d->n_pages > INT32_MAX / d->h_kv)
    return fail(GDN_ERR_UNSUPPORTED, "n_layers * n_pages * h_kv must stay below 2^31");
  // positions and lengths are int32 throughout
  if ((int64_t)d->max_pages * d->page_tokens > INT32_MAX - 256)
    return fail(GDN_ERR_UNSUPPORTED, "max_pages * page_tokens must stay below 2^31 - 256");
  return GDN_OK;
}

// The codes of one side as [blocks][page_tokens][d] bytes.
bool encode_codes(CUtensorMap *m, void *codes, const gdn_kv_desc &d) {
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      fn == nullptr || q != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return false;
  }
  const cuuint64_t dim = (cuuint64_t)d.d, rows = (cuuint64_t)d.page_tokens;
  cuuint64_t dims[3] = {dim, rows, (cuuint64_t)d.n_layers * d.n_pages * d.h_kv};
  cuuint64_t strides[2] = {dim, dim * rows};
  cuuint32_t box[3] = {(cuuint32_t)(d.d < 128 ? d.d : 128), 16, 1};
  cuuint32_t elem[3] = {1, 1, 1};
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)(
             m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             d.d < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Arguments that the three calls share.  On GDN_OK with *empty set there is
// nothing to do.
gdn_status check_call(const gdn_kv *c, int32_t layer, const int32_t *slot_ids,
                      const int32_t *starts, const int32_t *cu_seqlens, int32_t n_seqs,
                      int32_t total_tokens, const char *starts_name, bool *empty) {
  *empty = false;
  if (!c) return fail(GDN_ERR_ARG, "kv is NULL");
  if (layer < 0 || layer >= c->desc.n_layers)
    return fail(GDN_ERR_ARG, "layer %d outside [0, %d)", layer, c->desc.n_layers);
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != c->device)
    return fail(GDN_ERR_ARG, "current device %d is not the cache's device %d", dev, c->device);
  if (n_seqs < 0 || total_tokens < 0) return fail(GDN_ERR_ARG, "negative n_seqs/total_tokens");
  if (n_seqs > 65535) return fail(GDN_ERR_SIZE, "n_seqs = %d > 65535", n_seqs);
  if (!cu_seqlens && total_tokens != n_seqs)
    return fail(GDN_ERR_SIZE, "without cu_seqlens total_tokens must equal n_seqs");
  if (n_seqs == 0 || total_tokens == 0) {
    *empty = true;
    return GDN_OK;
  }
  if (!slot_ids || !starts) return fail(GDN_ERR_ARG, "slot_ids and %s must be non-NULL", starts_name);
  return GDN_OK;
}

// The caller's bound of the sequences' lengths, no larger than the call allows.
int32_t bound_seqlen(int32_t max_seqlen, const int32_t *cu_seqlens, int32_t total_tokens) {
  const int32_t most = cu_seqlens ? total_tokens : 1;
  return max_seqlen < 1 ? 1 : max_seqlen < most ? max_seqlen : most;
}

// Token rows: a stride of at least `width` elements, 16-byte aligned rows.
gdn_status check_rows(const void *p, int64_t *ld, int64_t width, gdn_dtype dt, const char *name) {
  if (*ld == 0) *ld = width;
  if (*ld < width)
    return fail(GDN_ERR_ARG, "%s: token stride %lld smaller than a token", name, (long long)*ld);
  if ((uintptr_t)p % 16 || (*ld * dtype_size(dt)) % 16)
    return fail(GDN_ERR_ARG, "%s rows must start 16-byte aligned", name);
  return GDN_OK;
}

// Host checks of the index arrays: slots in range (and distinct, when asked), cu_seqlens
// well-formed, the positions [first, last) of every sequence within a slot,
// and the pages that they lie on in range.  attend: starts are the lengths
// kv_lens and a sequence uses positions [0, kv_lens[i]); else they are pos and
// it uses [pos[i], pos[i] + len).
gdn_status check_index_arrays(const gdn_kv *c, const gdn::SeqIndex &seq, const int32_t *starts,
                              bool attend, bool distinct, cudaStream_t s) {
  const gdn_kv_desc &d = c->desc;
  std::vector<int32_t> slots, from, cu, table;
  gdn_status st;
  if ((st = fetch(slots, seq.slot_ids, (size_t)seq.n_seqs, s, "slot_ids")) ||
      (st = fetch(from, starts, (size_t)seq.n_seqs, s, attend ? "kv_lens" : "pos")) ||
      (st = fetch(table, c->view.table, (size_t)d.n_slots * d.max_pages, s, "page_table")))
    return st;
  if (seq.cu_seqlens) {
    if ((st = fetch(cu, seq.cu_seqlens, (size_t)seq.n_seqs + 1, s, "cu_seqlens"))) return st;
    if (cu[0] != 0) return fail(GDN_ERR_SIZE, "cu_seqlens[0] = %d, expected 0", cu[0]);
    for (int i = 0; i < seq.n_seqs; ++i)
      if (cu[i + 1] < cu[i]) return fail(GDN_ERR_SIZE, "cu_seqlens decreases at %d", i);
    if (cu[seq.n_seqs] != seq.total_tokens)
      return fail(GDN_ERR_SIZE, "cu_seqlens[%d] = %d, expected total_tokens %d", seq.n_seqs,
                  cu[seq.n_seqs], seq.total_tokens);
  }
  std::vector<unsigned char> seen((size_t)d.n_slots, 0);
  for (int i = 0; i < seq.n_seqs; ++i) {
    const int slot = slots[i];
    if (slot < 0 || slot >= d.n_slots)
      return fail(GDN_ERR_SLOT, "slot_ids[%d] = %d outside [0, %d)", i, slot, d.n_slots);
    if (distinct && seen[slot])
      return fail(GDN_ERR_DUP_SLOT, "slot id %d repeated (entry %d)", slot, i);
    seen[slot] = 1;
    const int64_t len = seq.cu_seqlens ? cu[i + 1] - cu[i] : 1;
    const int64_t a = attend ? 0 : from[i], b = attend ? from[i] : from[i] + len;
    if (a < 0 || b < 0 || b > c->view.capacity())
      return fail(GDN_ERR_SIZE, "%s[%d] = %d: outside the slot's %lld positions",
                  attend ? "kv_lens" : "pos", i, from[i], (long long)c->view.capacity());
    if (len == 0) continue;
    for (int64_t p = a / d.page_tokens; p * d.page_tokens < b; ++p) {
      const int32_t id = table[(size_t)slot * d.max_pages + p];
      if (id < 0 || id >= d.n_pages)
        return fail(GDN_ERR_SIZE, "page_table[%d][%lld] = %d outside [0, %d)", slot, (long long)p,
                    id, d.n_pages);
    }
  }
  return GDN_OK;
}

// No exception leaves a C entry point.
gdn_status check_index(const gdn_kv *c, const gdn::SeqIndex &seq, const int32_t *starts,
                       bool attend, bool distinct, cudaStream_t s) {
  try {
    return check_index_arrays(c, seq, starts, attend, distinct, s);
  } catch (const std::bad_alloc &) {
    return fail(GDN_ERR_SIZE, "no host memory to check the index arrays");
  }
}

}  // namespace

extern "C" {

size_t gdn_kv_code_bytes(const gdn_kv_desc *d) {
  if (!d || d->n_layers < 0 || d->n_pages < 0 || d->h_kv < 0 || d->page_tokens < 0 || d->d < 0)
    return 0;
  return (size_t)d->n_layers * d->n_pages * d->h_kv * d->page_tokens * d->d;
}

size_t gdn_kv_scale_bytes(const gdn_kv_desc *d) {
  if (!d || d->n_layers < 0 || d->n_pages < 0 || d->h_kv < 0) return 0;
  return (size_t)d->n_layers * d->n_pages * d->h_kv * sizeof(float);
}

gdn_status gdn_kv_create(const gdn_kv_desc *desc, void *k_codes, void *v_codes,
                         size_t code_bytes, float *k_scale, float *v_scale, size_t scale_bytes,
                         const int32_t *page_table, gdn_kv **out) {
  if (!out) return fail(GDN_ERR_ARG, "out is NULL");
  *out = nullptr;
  gdn_status st = check_desc(desc);
  if (st != GDN_OK) return st;
  if (!k_codes || !v_codes || !k_scale || !v_scale || !page_table)
    return fail(GDN_ERR_ARG, "codes, scales and page_table must be non-NULL");
  if ((uintptr_t)k_codes % 16 || (uintptr_t)v_codes % 16)
    return fail(GDN_ERR_ARG, "codes must be 16-byte aligned");
  if ((uintptr_t)k_scale % 4 || (uintptr_t)v_scale % 4 || (uintptr_t)page_table % 4)
    return fail(GDN_ERR_ARG, "scales and page_table must be 4-byte aligned");
  if (code_bytes < gdn_kv_code_bytes(desc))
    return fail(GDN_ERR_SIZE, "code_bytes %zu < %zu needed", code_bytes, gdn_kv_code_bytes(desc));
  if (scale_bytes < gdn_kv_scale_bytes(desc))
    return fail(GDN_ERR_SIZE, "scale_bytes %zu < %zu needed", scale_bytes,
                gdn_kv_scale_bytes(desc));
  int dev = -1, sm_count = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (desc->host_checks) {
    if ((st = check_device_ptr(k_codes, "k_codes")) || (st = check_device_ptr(v_codes, "v_codes")) ||
        (st = check_device_ptr(k_scale, "k_scale")) || (st = check_device_ptr(v_scale, "v_scale")) ||
        (st = check_device_ptr(page_table, "page_table")))
      return st;
  }
  e = cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(multiprocessor count)");
  gdn_kv *c = new (std::nothrow) gdn_kv;
  if (!c) return fail(GDN_ERR_SIZE, "no host memory for the handle");
  c->desc = *desc;
  c->device = dev;
  c->sm_count = sm_count;
  c->work.n = 0;
  if (!encode_codes(&c->k_map, k_codes, *desc) || !encode_codes(&c->v_map, v_codes, *desc)) {
    delete c;
    return fail(GDN_ERR_CUDA, "encoding the tensor maps of the codes failed");
  }
  unsigned int *err = nullptr;  // the error word, and the page calls' ticket
  e = cudaMalloc(&err, 2 * sizeof(*err));
  if (e == cudaSuccess) {
    e = cudaMemset(err, 0, 2 * sizeof(*err));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) cudaFree(err);
  }
  if (e != cudaSuccess) {
    delete c;
    return cuda_fail(e, "allocating the error word");
  }
  cudaMemPoolProps props = {};
  props.allocType = cudaMemAllocationTypePinned;
  props.location.type = cudaMemLocationTypeDevice;
  props.location.id = dev;
  e = cudaMemPoolCreate(&c->work.pool, &props);
  if (e == cudaSuccess) {
    uint64_t keep = UINT64_MAX;  // keep freed workspace for the next call
    e = cudaMemPoolSetAttribute(c->work.pool, cudaMemPoolAttrReleaseThreshold, &keep);
    if (e != cudaSuccess) cudaMemPoolDestroy(c->work.pool);
  }
  if (e != cudaSuccess) {
    cudaFree(err);
    delete c;
    return cuda_fail(e, "creating the workspace memory pool");
  }
  int log2 = 0;
  while ((1 << log2) < desc->page_tokens) ++log2;
  c->view = gdn::KVView{static_cast<uint8_t *>(k_codes), static_cast<uint8_t *>(v_codes), k_scale,
                        v_scale, page_table, err, desc->n_layers, desc->n_slots, desc->n_pages,
                        desc->max_pages, desc->page_tokens, log2, desc->h_q, desc->h_kv, desc->d,
                        desc->code, 0};
  *out = c;
  return ok();
}

gdn_status gdn_kv_destroy(gdn_kv *c) {
  if (!c) return ok();
  const OnDevice here(c->device);
  cudaError_t e = cudaDeviceSynchronize();
  if (here.status != cudaSuccess) e = here.status;
  cudaError_t e2 = cudaFree(c->view.err);
  for (int i = 0; i < c->work.n; ++i) {
    const cudaError_t ew = cudaFree(c->work.kept[i].mem);
    if (e2 == cudaSuccess) e2 = ew;
  }
  const cudaError_t e3 = cudaMemPoolDestroy(c->work.pool);
  if (e2 == cudaSuccess) e2 = e3;
  delete c;
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  if (e2 != cudaSuccess) return cuda_fail(e2, "releasing the cache handle");
  return ok();
}

gdn_status gdn_kv_get_error(gdn_kv *c, uint32_t *dev_err) {
  if (!c || !dev_err) return fail(GDN_ERR_ARG, "kv and dev_err must be non-NULL");
  unsigned int h = 0;
  const OnDevice here(c->device);
  cudaError_t e = here.status;
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&h, c->view.err, sizeof(h), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(c->view.err, 0, sizeof(h));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "reading the device error word");
  *dev_err = h;
  return ok();
}

gdn_status gdn_kv_set_test_flags(gdn_kv *c, uint32_t flags) {
  if (!c) return fail(GDN_ERR_ARG, "kv is NULL");
  if (flags & ~(uint32_t)GDN_TEST_KV_WAIT_TIMEOUT)
    return fail(GDN_ERR_ARG, "unknown test flags 0x%x", flags);
  c->view.test_flags = flags;
  return ok();
}

gdn_status gdn_kv_append(gdn_kv *c, int32_t layer, const int32_t *slot_ids, const int32_t *pos,
                         const int32_t *cu_seqlens, int32_t n_seqs, int32_t total_tokens,
                         int32_t max_seqlen, const void *k, int64_t ld_k, const void *v,
                         int64_t ld_v, gdn_dtype dtype, gdn_stream stream) {
  bool empty;
  gdn_status st = check_call(c, layer, slot_ids, pos, cu_seqlens, n_seqs, total_tokens, "pos",
                             &empty);
  if (st != GDN_OK) return st;
  if (!dtype_ok(dtype)) return fail(GDN_ERR_DTYPE, "k/v dtype must be F32 or BF16");
  if (empty) return ok();
  if (!k || !v) return fail(GDN_ERR_ARG, "k and v must be non-NULL");
  const int64_t width = (int64_t)c->desc.h_kv * c->desc.d;
  if ((st = check_rows(k, &ld_k, width, dtype, "k")) ||
      (st = check_rows(v, &ld_v, width, dtype, "v")))
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const gdn::SeqIndex seq{slot_ids, cu_seqlens, n_seqs, total_tokens};
  if (c->desc.host_checks &&
      ((st = check_index(c, seq, pos, false, true, s)) || (st = check_device_ptr(k, "k")) ||
       (st = check_device_ptr(v, "v"))))
    return st;
  const gdn::KVRows rows{const_cast<void *>(k), const_cast<void *>(v), ld_k, ld_v, dtype};
  max_seqlen = bound_seqlen(max_seqlen, cu_seqlens, total_tokens);
  const cudaError_t e = gdn::launch_kv_append(c->view, layer, seq, pos, max_seqlen, rows, s);
  if (e != cudaSuccess) return cuda_fail(e, "KV append launch");
  return ok();
}

gdn_status gdn_kv_read(gdn_kv *c, int32_t layer, const int32_t *slot_ids, const int32_t *pos,
                       const int32_t *cu_seqlens, int32_t n_seqs, int32_t total_tokens,
                       int32_t max_seqlen, void *k, int64_t ld_k, void *v, int64_t ld_v,
                       gdn_dtype dtype, gdn_stream stream) {
  bool empty;
  gdn_status st = check_call(c, layer, slot_ids, pos, cu_seqlens, n_seqs, total_tokens, "pos",
                             &empty);
  if (st != GDN_OK) return st;
  if (!dtype_ok(dtype)) return fail(GDN_ERR_DTYPE, "k/v dtype must be F32 or BF16");
  if (empty) return ok();
  if (!k && !v) return fail(GDN_ERR_ARG, "k and v are both NULL");
  const int64_t width = (int64_t)c->desc.h_kv * c->desc.d;
  if ((st = check_rows(k, &ld_k, width, dtype, "k")) ||
      (st = check_rows(v, &ld_v, width, dtype, "v")))
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const gdn::SeqIndex seq{slot_ids, cu_seqlens, n_seqs, total_tokens};
  if (c->desc.host_checks &&
      ((st = check_index(c, seq, pos, false, false, s)) || (k && (st = check_device_ptr(k, "k"))) ||
       (v && (st = check_device_ptr(v, "v")))))
    return st;
  const gdn::KVRows rows{k, v, ld_k, ld_v, dtype};
  max_seqlen = bound_seqlen(max_seqlen, cu_seqlens, total_tokens);
  const cudaError_t e = gdn::launch_kv_read(c->view, layer, seq, pos, max_seqlen, rows, s);
  if (e != cudaSuccess) return cuda_fail(e, "KV read launch");
  return ok();
}

gdn_status gdn_kv_attend(gdn_kv *c, int32_t layer, const int32_t *slot_ids,
                         const int32_t *kv_lens, const int32_t *cu_seqlens, int32_t n_seqs,
                         int32_t total_tokens, int32_t max_seqlen, int32_t max_kv_len,
                         const void *q, int64_t ld_q, gdn_dtype q_dtype, void *o, int64_t ld_o,
                         gdn_dtype o_dtype, float scale, gdn_stream stream) {
  bool empty;
  gdn_status st = check_call(c, layer, slot_ids, kv_lens, cu_seqlens, n_seqs, total_tokens,
                             "kv_lens", &empty);
  if (st != GDN_OK) return st;
  if (!dtype_ok(q_dtype) || !dtype_ok(o_dtype))
    return fail(GDN_ERR_DTYPE, "q and o dtypes must be F32 or BF16");
  if (!std::isfinite(scale)) return fail(GDN_ERR_ARG, "scale is not finite");
  if (empty) return ok();
  if (!q || !o) return fail(GDN_ERR_ARG, "q and o must be non-NULL");
  const int64_t width = (int64_t)c->desc.h_q * c->desc.d;
  if ((st = check_rows(q, &ld_q, width, q_dtype, "q")) ||
      (st = check_rows(o, &ld_o, width, o_dtype, "o")))
    return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const gdn::SeqIndex seq{slot_ids, cu_seqlens, n_seqs, total_tokens};
  if (c->desc.host_checks &&
      ((st = check_index(c, seq, kv_lens, true, false, s)) || (st = check_device_ptr(q, "q")) ||
       (st = check_device_ptr(o, "o"))))
    return st;
  const int64_t capacity = c->view.capacity();
  const int32_t hint = max_kv_len < 1 ? 1 : max_kv_len;
  const gdn::KVAttendArgs a{seq,  kv_lens, bound_seqlen(max_seqlen, cu_seqlens, total_tokens),
                            hint < capacity ? hint : (int)capacity, hint, q, o, ld_q, ld_o,
                            q_dtype, o_dtype, scale};
  const gdn::KVHost h{&c->k_map, &c->v_map, c->sm_count, c->device, &c->work};
  const cudaError_t e = gdn::launch_kv_attend(c->view, layer, a, h, s);
  if (e != cudaSuccess) return cuda_fail(e, "KV attention launch");
  return ok();
}

}  // extern "C"
