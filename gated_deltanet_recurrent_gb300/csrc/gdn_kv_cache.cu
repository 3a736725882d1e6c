// Writing the 8-bit KV cache and reading it back.
//
// Append.  The unit is one (page, KV head, side) block: its scale 2^e comes
// from the largest finite magnitude of the new tokens that fall into it (and
// from its old scale, where it keeps earlier tokens), and every code is
// value * 2^-e rounded once to nearest even -- the product by a power of two is
// exact.  Both kernels are HBM-bound: the new rows are read once, one byte is
// written per element.
//   tile kernel (prompts): one CTA per block; the block's new rows stay in
//     registers (32 per thread) between the maximum and the codes.
//   warp kernel (single tokens and drafts): one warp per (sequence, head,
//     side), which walks its pages in order; there is little to read, so what
//     counts is the chain of dependent loads (slot -> page -> scale) and the
//     number of warps that hide it.  The rows are read twice, the second time
//     from L1.
// A page is written by one sequence of a call, so no two units meet.  Measured,
// append and read-back together: 8192 float32 tokens of 8 x 128 (168 MB) 42 us,
// 4.0 TB/s; 8 pieces of up to 2048 bf16 tokens of 2 x 256 (59 MB) 20 us, of
// which a third is the chain of loads at each kernel's start.  Each alone, on
// inputs out of L2: 28 and 26 us, 17.5 and 15.5 us, a step of 512 tokens of 8 x
// 128 11.4 and 17.5 us (28 MB read back).  Below some MB a call costs what its
// launch does.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

// Token range and first position of sequence i; false: nothing to do (an
// error bit is set where the entry is bad; `report`: this thread reports).  All
// loads are issued before the first check.
__device__ __forceinline__ bool kv_sequence(const KVView &c, const SeqIndex &seq,
                                            const int32_t *pos, int i, bool report, int *slot,
                                            int *tok0, int *len, int *first) {
  *slot = seq.slot_ids[i];
  *first = pos[i];
  *tok0 = i;
  int hi = i + 1;
  if (seq.cu_seqlens != nullptr) {
    *tok0 = seq.cu_seqlens[i];
    hi = seq.cu_seqlens[i + 1];
  }
  *len = hi - *tok0;
  if (*slot < 0 || *slot >= c.n_slots) {
    if (report) raise_error(c.err, GDN_DEVERR_SLOT);
    return false;
  }
  if (*tok0 < 0 || hi < *tok0 || hi > seq.total_tokens || *first < 0 ||
      (int64_t)*first + *len > c.capacity()) {
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

// 16 bytes of a row, as they lie: 4 or 8 elements.  A lane's neighbours take the
// next ones, so that loads, codes and values all go in whole sectors.
template <typename T>
constexpr int kElems = 16 / sizeof(T);

// Largest magnitude as float32 bits, which order like the magnitudes: infinities
// (0x7f800000) above the finite ones, NaN above those.
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint4 r, uint32_t m) {
  if constexpr (sizeof(T) == 4) {
    m = max(max(m, r.x & 0x7fffffffu), max(r.y & 0x7fffffffu, r.z & 0x7fffffffu));
    return max(m, r.w & 0x7fffffffu);
  } else {
    const uint32_t x = __vmaxu2(__vmaxu2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                                __vmaxu2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu));
    return max(m, max(x << 16, x & 0x7fff0000u));
  }
}

template <typename T>
__device__ __forceinline__ void widen(uint4 r, float *x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (sizeof(T) == 4) {
      x[j] = __uint_as_float(w[j]);
    } else {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The same over the finite elements only (for blocks that hold others).
template <typename T>
__device__ __forceinline__ uint32_t finite_max_bits(uint4 r, uint32_t m) {
  float x[kElems<T>];
  widen<T>(r, x);
#pragma unroll
  for (int j = 0; j < kElems<T>; ++j) {
    const uint32_t b = __float_as_uint(x[j]) & 0x7fffffffu;
    if (b < kInfBits) m = max(m, b);
  }
  return m;
}

// The codes of 16 bytes of elements; `odd`: NaN may be among them, and is stored as zero.
template <int CODE, typename T>
__device__ __forceinline__ void store_codes(uint8_t *p, uint4 r, float inv, bool odd) {
  using C = kv::Code<CODE>;
  float x[kElems<T>];
  widen<T>(r, x);
#pragma unroll
  for (int j = 0; j < kElems<T>; ++j) {
    x[j] *= inv;
    if (odd && x[j] != x[j]) x[j] = 0.f;
  }
  const uint32_t lo = C::encode4(x[0], x[1], x[2], x[3]);
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<uint32_t *>(p) = lo;
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(lo, C::encode4(x[4], x[5], x[6], x[7]));
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

// ---- prompts: a CTA per block, with the block's elements in its registers ----

constexpr int kVec = 8;  // 16-byte vectors per thread

template <typename T, int CODE>
__global__ void __launch_bounds__(sizeof(T) == 2 ? 512 : 1024, sizeof(T) == 2 ? 2 : 1)
    append_tile_kernel(KVView c, int layer, SeqIndex seq, const int32_t *__restrict__ pos,
                       KVRows rows) {
  __shared__ uint32_t s_max[2][32];
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
  // vectors of a row, a power of two
  const int dv_log2 = 31 - __clz(c.d / kElems<T>), dv = 1 << dv_log2;
  // the largest of the CTA's `m`
  auto reduce = [&](uint32_t m, int buf) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (nt > 32) {
      if ((tid & 31) == 0) s_max[buf][tid >> 5] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, (tid & 31) < (nt >> 5) ? s_max[buf][tid & 31] : 0u);
    }
    return m;
  };
  // the grid's x covers max_seqlen; a sequence that is longer than that takes more rounds
  for (int pg = page0 + blockIdx.x; pg <= page1; pg += gridDim.x) {
    const int start = pg << c.page_log2;
    const int off = pg == page0 ? first - start : 0;
    const int end = min(c.page_tokens, first + len - start);
    const T *base = src + (int64_t)(tok0 + start + off - first) * ld;
    const int nv = (end - off) * dv;
    auto vec = [&](int v) {
      return *reinterpret_cast<const uint4 *>(base + (int64_t)(v >> dv_log2) * ld +
                                              (v & (dv - 1)) * kElems<T>);
    };
    // the elements are on their way before the page id and the scale are asked for
    uint4 x[kVec];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = i * nt + tid;
      if (v < nv) x[i] = vec(v);
    }
    const int id = kv_page(c, slot, pg, blockIdx.y + tid == 0);
    if (id < 0) continue;
    const int64_t blk = c.block(layer, id, head);
    uint8_t *codes = (side ? c.v : c.k) + (blk << c.page_log2) * c.d;
    float *scale = (side ? c.v_scale : c.k_scale) + blk;
    const float was = off > 0 ? *scale : 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i * nt + tid < nv) m = max_bits<T>(x[i], m);
    m = reduce(m, 0);
    const bool odd = m >= kInfBits;
    if (odd) {
      if (tid == 0) raise_error(c.err, GDN_DEVERR_VALUE);
      m = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (i * nt + tid < nv) m = finite_max_bits<T>(x[i], m);
      m = reduce(m, 1);
    }
    int e = kv::Code<CODE>::exponent(__uint_as_float(m));
    if (off > 0) {
      const int old = kv::scale_exponent<CODE>(was);
      if (e > old)
        rescale<CODE>(codes, off * c.d, kv::pow2f(max(old - e, -126)), tid, nt);
      else
        e = old;
    }
    const float inv = kv::pow2f(-e);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int v = i * nt + tid;
      if (v < nv) store_codes<CODE, T>(codes + off * c.d + v * kElems<T>, x[i], inv, odd);
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
  const int dv_log2 = 31 - __clz(c.d / kElems<T>), dv = 1 << dv_log2;
  for (int done = 0; done < len;) {
    const int at = first + done, off = at & (c.page_tokens - 1);
    const int take = min(len - done, c.page_tokens - off);
    const T *base = src + (int64_t)(tok0 + done) * ld;
    const int nv = take * dv;
    auto vec = [&](int v) {
      return *reinterpret_cast<const uint4 *>(base + (int64_t)(v >> dv_log2) * ld +
                                              (v & (dv - 1)) * kElems<T>);
    };
    // a token's elements (one vector per lane) are on their way before the page id is asked for
    uint4 x;
    if (lane < nv) x = vec(lane);
    const int id = kv_page(c, slot, at >> c.page_log2, r + lane == 0);
    done += take;
    if (id < 0) continue;
    const int64_t blk = c.block(layer, id, head);
    uint8_t *codes = (side ? c.v : c.k) + (blk << c.page_log2) * c.d;
    float *scale = (side ? c.v_scale : c.k_scale) + blk;
    const float was = off > 0 ? *scale : 0.f;
    uint32_t m = 0;
    if (lane < nv) m = max_bits<T>(x, m);
    for (int v = lane + 32; v < nv; v += 32) m = max_bits<T>(vec(v), m);
    m = __reduce_max_sync(0xffffffffu, m);
    const bool odd = m >= kInfBits;
    if (odd) {
      if (lane == 0) raise_error(c.err, GDN_DEVERR_VALUE);
      m = 0;
      for (int v = lane; v < nv; v += 32) m = finite_max_bits<T>(vec(v), m);
      m = __reduce_max_sync(0xffffffffu, m);
    }
    int e = kv::Code<CODE>::exponent(__uint_as_float(m));
    if (off > 0) {
      const int old = kv::scale_exponent<CODE>(was);
      if (e > old)
        rescale<CODE>(codes, off * c.d, kv::pow2f(max(old - e, -126)), lane, 32);
      else
        e = old;
    }
    const float inv = kv::pow2f(-e);
    if (lane < nv) store_codes<CODE, T>(codes + off * c.d + lane * kElems<T>, x, inv, odd);
    for (int v = lane + 32; v < nv; v += 32)
      store_codes<CODE, T>(codes + off * c.d + v * kElems<T>, vec(v), inv, odd);
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = kv::pow2f(e);
  }
}

// ---- read back ----
//
// A thread writes 16 bytes of each of kReadItems places; the page ids of all of
// them are asked for at once, then the codes and scales of all.

constexpr int kReadThreads = 256;
constexpr int kReadItems = 4;

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
  constexpr int E = kElems<T>;
  const int dv_log2 = 31 - __clz(c.d / E), per_token = c.h_kv << dv_log2;
  const int64_t total = (int64_t)len * per_token;
  for (int64_t u0 = (int64_t)blockIdx.x * (kReadThreads * kReadItems) + threadIdx.x; u0 < total;
       u0 += (int64_t)gridDim.x * (kReadThreads * kReadItems)) {
    int t[kReadItems], r[kReadItems], id[kReadItems];
#pragma unroll
    for (int x = 0; x < kReadItems; ++x) {
      const int64_t u = u0 + x * kReadThreads;
      id[x] = -1;
      if (u < total) {
        t[x] = u >> 32 == 0 ? (int)((uint32_t)u / (uint32_t)per_token) : (int)(u / per_token);
        r[x] = (int)(u - (int64_t)t[x] * per_token);
        id[x] = kv_page(c, slot, (first + t[x]) >> c.page_log2, true);
      }
    }
    uint32_t w[kReadItems][E / 4];
    float f[kReadItems];
#pragma unroll
    for (int x = 0; x < kReadItems; ++x)
      if (id[x] >= 0) {
        const int head = r[x] >> dv_log2, row = (first + t[x]) & (c.page_tokens - 1);
        const int64_t blk = c.block(layer, id[x], head);
        const uint8_t *p = codes + ((blk << c.page_log2) + row) * c.d +
                           E * (r[x] - (head << dv_log2));
        if constexpr (E == 4) {
          w[x][0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
          const uint2 two = *reinterpret_cast<const uint2 *>(p);
          w[x][0] = two.x, w[x][E / 4 - 1] = two.y;
        }
        f[x] = scale[blk];
      }
#pragma unroll
    for (int x = 0; x < kReadItems; ++x)
      if (id[x] >= 0) {
        T *dst = out + (int64_t)(tok0 + t[x]) * ld + (int64_t)E * r[x];
        const float4 a = scale4(f[x], kv::Code<CODE>::decode4(w[x][0]));
        if constexpr (E == 4) {
          *reinterpret_cast<float4 *>(dst) = a;
        } else {
          const float4 b = scale4(f[x], kv::Code<CODE>::decode4(w[x][E / 4 - 1]));
          const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(a.x, a.y),
                                       __floats2bfloat162_rn(a.z, a.w),
                                       __floats2bfloat162_rn(b.x, b.y),
                                       __floats2bfloat162_rn(b.z, b.w)};
          *reinterpret_cast<uint4 *>(dst) = *reinterpret_cast<const uint4 *>(h);
        }
      }
  }
}

template <typename T, int CODE>
cudaError_t append_t(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                     int max_seqlen, const KVRows &rows, cudaStream_t s) {
  if (max_seqlen <= 8) {
    const int64_t units = (int64_t)seq.n_seqs * 2 * c.h_kv;
    return kv::launch(append_warp_kernel<T, CODE>,
                      dim3((unsigned)((units + kAppendWarps - 1) / kAppendWarps)),
                      32 * kAppendWarps, 0, s, 1, c, layer, seq, pos, rows);
  }
  const int vecs = c.page_tokens * c.d / (kElems<T> * kVec), threads = vecs < 32 ? 32 : vecs;
  // an unaligned range of max_seqlen tokens touches one page more than an aligned one
  const int64_t pages = ((int64_t)max_seqlen + c.page_tokens - 2) / c.page_tokens + 1;
  dim3 grid((unsigned)(pages < c.max_pages ? pages : c.max_pages), (unsigned)(2 * c.h_kv),
            (unsigned)seq.n_seqs);
  return kv::launch(append_tile_kernel<T, CODE>, grid, threads, 0, s, 1, c, layer, seq, pos, rows);
}

template <typename T, int CODE>
cudaError_t read_t(const KVView &c, int layer, const SeqIndex &seq, const int32_t *pos,
                   int max_seqlen, const KVRows &rows, cudaStream_t s) {
  const int64_t work = (int64_t)max_seqlen * c.h_kv * (c.d / kElems<T>);
  int64_t bx = (work + kReadThreads * kReadItems - 1) / (kReadThreads * kReadItems);
  if (bx > 65535) bx = 65535;
  return kv::launch(read_kernel<T, CODE>, dim3((unsigned)bx, 2, (unsigned)seq.n_seqs),
                    kReadThreads, 0, s, 1, c, layer, seq, pos, rows);
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
