// Writing the 8-bit KV cache and reading it back.
//
// Append.  The unit is one (page, KV head, side) block: its scale 2^e comes
// from the largest finite magnitude of the new tokens that fall into it (and
// from its old scale, where it keeps earlier tokens), and every code is
// value * 2^-e rounded once to nearest even -- the product by a power of two is
// exact.  Both kernels are HBM-bound: the new rows are read once, one byte is
// written per element.
//   tile kernel (prompts): one CTA per block; the block's new rows stay in
//     registers (64 elements per thread) between the maximum and the codes.
//   warp kernel (single tokens and drafts): one warp per (sequence, head,
//     side), which walks its pages in order; there is little to read, so what
//     counts is the chain of dependent loads (slot -> page -> scale) and the
//     number of warps that hide it.  The rows are read twice, the second time
//     from L1.
// A page is written by one sequence of a call, so no two units meet.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

// Token range and first position of sequence i; false: nothing to do (an
// error bit is set where the entry is bad; `report`: this thread reports).
__device__ __forceinline__ bool kv_sequence(const KVView &c, const SeqIndex &seq,
                                            const int32_t *pos, int i, bool report, int *slot,
                                            int *tok0, int *len, int *first) {
  *slot = seq.slot_ids[i];
  if (*slot < 0 || *slot >= c.n_slots) {
    if (report) raise_error(c.err, GDN_DEVERR_SLOT);
    return false;
  }
  *tok0 = i;
  *len = 1;
  if (seq.cu_seqlens != nullptr) {
    *tok0 = seq.cu_seqlens[i];
    const int hi = seq.cu_seqlens[i + 1];
    if (*tok0 < 0 || hi < *tok0 || hi > seq.total_tokens) {
      if (report) raise_error(c.err, GDN_DEVERR_SEQ);
      return false;
    }
    *len = hi - *tok0;
  }
  *first = pos[i];
  if (*first < 0 || (int64_t)*first + *len > c.capacity()) {
    if (report) raise_error(c.err, GDN_DEVERR_SEQ);
    return false;
  }
  return *len > 0;
}

// A page id of the table, or -1 (reported) if it is out of range.
__device__ __forceinline__ int kv_page(const KVView &c, int slot, int index, bool report) {
  const int id = c.table[(int64_t)slot * c.max_pages + index];
  if (id >= 0 && id < c.n_pages) return id;
  if (report) raise_error(c.err, GDN_DEVERR_PAGE);
  return -1;
}

// Eight consecutive elements of a row (16-byte aligned), NaN as zero; *odd is
// set where one is not finite.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float *x, bool *odd) {
  const float4 a = Elem<T>::load4(p), b = Elem<T>::load4(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!(fabsf(x[j]) <= 3.402823466e38f)) {
      *odd = true;
      if (x[j] != x[j]) x[j] = 0.f;
    }
  }
}

__device__ __forceinline__ float finite_max8(const float *x, float m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(x[j]);
    if (a <= 3.402823466e38f) m = fmaxf(m, a);
  }
  return m;
}

template <int CODE>
__device__ __forceinline__ void store8(uint8_t *p, const float *x, float inv) {
  using C = kv::Code<CODE>;
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(C::encode4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                 C::encode4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// codes [0, bytes) of a block times `ratio` (a power of two below one)
template <int CODE>
__device__ __forceinline__ void rescale(uint8_t *block, int bytes, float ratio, int t, int threads) {
  using C = kv::Code<CODE>;
  for (int i = t * 16; i < bytes; i += threads * 16) {
    uint4 w = *reinterpret_cast<uint4 *>(block + i);
    uint32_t *v = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = C::decode4(v[j]);
      v[j] = C::encode4(x.x * ratio, x.y * ratio, x.z * ratio, x.w * ratio);
    }
    *reinterpret_cast<uint4 *>(block + i) = w;
  }
}

// ---- prompts: a CTA of max(32, page_tokens * d / 64) threads per block ----

constexpr int kVec = 8;  // vectors of 8 elements per thread

template <typename T, int CODE>
__global__ void __launch_bounds__(512)
    append_tile_kernel(KVView c, int layer, SeqIndex seq, const int32_t *__restrict__ pos,
                       KVRows rows) {
  __shared__ float s_max[16];
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
  const int tid = threadIdx.x, nt = blockDim.x;
  int slot, tok0, len, first;
  if (!kv_sequence(c, seq, pos, blockIdx.z, blockIdx.x + blockIdx.y + tid == 0, &slot, &tok0,
                   &len, &first))
    return;
  const int page0 = first >> c.page_log2, page1 = (first + len - 1) >> c.page_log2;
  const int64_t ld = side ? rows.ld_v : rows.ld_k;
  const T *src = static_cast<const T *>(side ? rows.v : rows.k) + (int64_t)head * c.d;
  const int d8 = c.d >> 3;
  // the grid's x covers max_seqlen; a sequence that is longer than that takes more rounds
  for (int pg = page0 + blockIdx.x; pg <= page1; pg += gridDim.x) {
    const int id = kv_page(c, slot, pg, blockIdx.y + tid == 0);
    if (id < 0) continue;
    const int start = pg << c.page_log2;
    const int off = pg == page0 ? first - start : 0;
    const int end = min(c.page_tokens, first + len - start);
    const T *base = src + (int64_t)(tok0 + start + off - first) * ld;
    const int nv = (end - off) * d8;
    float x[kVec][8];
    bool odd = false;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = i * nt + tid;
      if (v < nv) {
        load8<T>(base + (int64_t)(v / d8) * ld + (v % d8) * 8, x[i], &odd);
        m = finite_max8(x[i], m);
      }
    }
    if (odd) raise_error(c.err, GDN_DEVERR_VALUE);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (nt > 32) {
      if ((tid & 31) == 0) s_max[tid >> 5] = m;
      __syncthreads();
      for (int w = 0; w < nt >> 5; ++w) m = fmaxf(m, s_max[w]);
    }
    const int64_t blk = c.block(layer, id, head);
    uint8_t *codes = (side ? c.v : c.k) + (blk << c.page_log2) * c.d;
    float *scale = (side ? c.v_scale : c.k_scale) + blk;
    int e = kv::Code<CODE>::exponent(m);
    if (off > 0) {
      const int old = kv::scale_exponent<CODE>(*scale);
      if (e > old)
        rescale<CODE>(codes, off * c.d, kv::pow2f(max(old - e, -126)), tid, nt);
      else
        e = old;
    }
    const float inv = kv::pow2f(-e);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = i * nt + tid;
      if (v < nv) store8<CODE>(codes + (int64_t)off * c.d + v * 8, x[i], inv);
    }
    __syncthreads();  // every thread has read the old scale and s_max
    if (tid == 0) *scale = kv::pow2f(e);
  }
}

// ---- single tokens and drafts: a warp per (sequence, head, side) ----

constexpr int kAppendWarps = 4;

template <typename T, int CODE>
__global__ void __launch_bounds__(32 * kAppendWarps)
    append_warp_kernel(KVView c, int layer, SeqIndex seq, const int32_t *__restrict__ pos,
                       KVRows rows) {
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int per_seq = 2 * c.h_kv;
  if (unit >= (int64_t)seq.n_seqs * per_seq) return;
  const int i = (int)(unit / per_seq), r = (int)(unit % per_seq);
  const int head = r >> 1, side = r & 1;
  int slot, tok0, len, first;
  if (!kv_sequence(c, seq, pos, i, r + lane == 0, &slot, &tok0, &len, &first)) return;
  const int64_t ld = side ? rows.ld_v : rows.ld_k;
  const T *src = static_cast<const T *>(side ? rows.v : rows.k) + (int64_t)head * c.d;
  const int d8 = c.d >> 3;
  for (int done = 0; done < len;) {
    const int at = first + done, off = at & (c.page_tokens - 1);
    const int take = min(len - done, c.page_tokens - off);
    const T *base = src + (int64_t)(tok0 + done) * ld;
    const int id = kv_page(c, slot, at >> c.page_log2, r + lane == 0);
    done += take;
    if (id < 0) continue;
    const int64_t blk = c.block(layer, id, head);
    uint8_t *codes = (side ? c.v : c.k) + (blk << c.page_log2) * c.d;
    float *scale = (side ? c.v_scale : c.k_scale) + blk;
    const float was = off > 0 ? *scale : 0.f;
    const int nv = take * d8;
    float x[8];
    bool odd = false;
    float m = 0.f;
    for (int v = lane; v < nv; v += 32) {
      load8<T>(base + (int64_t)(v / d8) * ld + (v % d8) * 8, x, &odd);
      m = finite_max8(x, m);
    }
    if (odd) raise_error(c.err, GDN_DEVERR_VALUE);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    int e = kv::Code<CODE>::exponent(m);
    if (off > 0) {
      const int old = kv::scale_exponent<CODE>(was);
      if (e > old)
        rescale<CODE>(codes, off * c.d, kv::pow2f(max(old - e, -126)), lane, 32);
      else
        e = old;
    }
    const float inv = kv::pow2f(-e);
    for (int v = lane; v < nv; v += 32) {
      if (nv > 32) load8<T>(base + (int64_t)(v / d8) * ld + (v % d8) * 8, x, &odd);
      store8<CODE>(codes + (int64_t)off * c.d + v * 8, x, inv);
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = kv::pow2f(e);
  }
}

// ---- read back: a thread per 16 codes ----

constexpr int kReadThreads = 256;

template <typename T>
__device__ __forceinline__ void put4(T *p, float4 v);
template <>
__device__ __forceinline__ void put4<float>(float *p, float4 v) {
  *reinterpret_cast<float4 *>(p) = v;
}
template <>
__device__ __forceinline__ void put4<bf16>(bf16 *p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

template <typename T, int CODE>
__global__ void __launch_bounds__(kReadThreads)
    read_kernel(KVView c, int layer, SeqIndex seq, const int32_t *__restrict__ pos, KVRows rows) {
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int side = blockIdx.y;
  if ((side ? rows.v : rows.k) == nullptr) return;
  int slot, tok0, len, first;
  if (!kv_sequence(c, seq, pos, blockIdx.z, blockIdx.x + blockIdx.y + threadIdx.x == 0, &slot,
                   &tok0, &len, &first))
    return;
  const uint8_t *codes = side ? c.v : c.k;
  const float *scale = side ? c.v_scale : c.k_scale;
  T *out = static_cast<T *>(side ? rows.v : rows.k);
  const int64_t ld = side ? rows.ld_v : rows.ld_k;
  const int d16 = c.d >> 4, per_token = c.h_kv * d16;
  const int64_t total = (int64_t)len * per_token;
  for (int64_t u = (int64_t)blockIdx.x * kReadThreads + threadIdx.x; u < total;
       u += (int64_t)gridDim.x * kReadThreads) {
    const int t = (int)(u / per_token), r = (int)(u % per_token);
    const int head = r / d16, j = r % d16, at = first + t;
    const int id = kv_page(c, slot, at >> c.page_log2, true);
    if (id < 0) continue;
    const int64_t blk = c.block(layer, id, head);
    const int row = at & (c.page_tokens - 1);
    const uint4 w = *reinterpret_cast<const uint4 *>(
        codes + ((blk << c.page_log2) + row) * c.d + 16 * j);
    const float f = scale[blk];
    T *dst = out + (int64_t)(tok0 + t) * ld + (int64_t)head * c.d + 16 * j;
    put4<T>(dst, scale4(f, kv::Code<CODE>::decode4(w.x)));
    put4<T>(dst + 4, scale4(f, kv::Code<CODE>::decode4(w.y)));
    put4<T>(dst + 8, scale4(f, kv::Code<CODE>::decode4(w.z)));
    put4<T>(dst + 12, scale4(f, kv::Code<CODE>::decode4(w.w)));
  }
}

template <typename T, int CODE>
cudaError_t append_t(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                     int max_seqlen, const KVRows &rows, cudaStream_t s) {
  if (max_seqlen <= 8) {
    const int64_t units = (int64_t)seq.n_seqs * 2 * c.h_kv;
    return kv::launch(append_warp_kernel<T, CODE>,
                      dim3((unsigned)((units + kAppendWarps - 1) / kAppendWarps)),
                      32 * kAppendWarps, 0, s, c, layer, seq, pos, rows);
  }
  const int threads = c.page_tokens * c.d / (8 * kVec) < 32 ? 32 : c.page_tokens * c.d / (8 * kVec);
  // an unaligned range of max_seqlen tokens touches one page more than an aligned one
  const int64_t pages = ((int64_t)max_seqlen + c.page_tokens - 2) / c.page_tokens + 1;
  dim3 grid((unsigned)(pages < c.max_pages ? pages : c.max_pages), (unsigned)(2 * c.h_kv),
            (unsigned)seq.n_seqs);
  return kv::launch(append_tile_kernel<T, CODE>, grid, threads, 0, s, c, layer, seq, pos, rows);
}

template <typename T, int CODE>
cudaError_t read_t(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                   int max_seqlen, const KVRows &rows, cudaStream_t s) {
  const int64_t work = (int64_t)max_seqlen * c.h_kv * (c.d / 16);
  int64_t bx = (work + kReadThreads - 1) / kReadThreads;
  if (bx > 65535) bx = 65535;
  return kv::launch(read_kernel<T, CODE>, dim3((unsigned)bx, 2, (unsigned)seq.n_seqs),
                    kReadThreads, 0, s, c, layer, seq, pos, rows);
}

}  // namespace

cudaError_t launch_kv_append(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                             int max_seqlen, const KVRows &rows, cudaStream_t s) {
  const bool f32 = rows.dtype == GDN_F32;
  if (c.code == GDN_KV_I8)
    return f32 ? append_t<float, GDN_KV_I8>(c, layer, seq, pos, max_seqlen, rows, s)
               : append_t<bf16, GDN_KV_I8>(c, layer, seq, pos, max_seqlen, rows, s);
  return f32 ? append_t<float, GDN_KV_E4M3>(c, layer, seq, pos, max_seqlen, rows, s)
             : append_t<bf16, GDN_KV_E4M3>(c, layer, seq, pos, max_seqlen, rows, s);
}

cudaError_t launch_kv_read(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                           int max_seqlen, const KVRows &rows, cudaStream_t s) {
  const bool f32 = rows.dtype == GDN_F32;
  if (c.code == GDN_KV_I8)
    return f32 ? read_t<float, GDN_KV_I8>(c, layer, seq, pos, max_seqlen, rows, s)
               : read_t<bf16, GDN_KV_I8>(c, layer, seq, pos, max_seqlen, rows, s);
  return f32 ? read_t<float, GDN_KV_E4M3>(c, layer, seq, pos, max_seqlen, rows, s)
             : read_t<bf16, GDN_KV_E4M3>(c, layer, seq, pos, max_seqlen, rows, s);
}

}  // namespace gdn
