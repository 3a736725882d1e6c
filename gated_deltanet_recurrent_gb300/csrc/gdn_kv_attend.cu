// Causal grouped-query attention over the 8-bit KV cache, in its plain form:
// a warp per (query token, query head) walks the cached positions in order
// with the running maximum and sum of the softmax, d / 32 elements of the
// query, the key and the accumulator per lane.
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;

template <int CODE, int D, typename TQ, typename TO>
__global__ void __launch_bounds__(32 * kWarps)
    attend_plain_kernel(KVView c, int layer, KVAttendArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, i = blockIdx.y;
  const bool report = blockIdx.x + threadIdx.x == 0;
  const int slot = a.seq.slot_ids[i];
  if (slot < 0 || slot >= c.n_slots) {
    if (report) raise_error(c.err, GDN_DEVERR_SLOT);
    return;
  }
  int lo = i, len = 1;
  if (a.seq.cu_seqlens != nullptr) {
    lo = a.seq.cu_seqlens[i];
    const int hi = a.seq.cu_seqlens[i + 1];
    if (lo < 0 || hi < lo || hi > a.seq.total_tokens) {
      if (report) raise_error(c.err, GDN_DEVERR_SEQ);
      return;
    }
    len = hi - lo;
  }
  const int kv_len = a.kv_lens[i];
  if (kv_len < 0 || kv_len > c.capacity()) {
    if (report) raise_error(c.err, GDN_DEVERR_SEQ);
    return;
  }
  const int64_t rows = (int64_t)len * c.h_q;
  for (int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * kWarps) {
    const int t = (int)(r / c.h_q), h = (int)(r % c.h_q), hk = h / (c.h_q / c.h_kv);
    const TQ *q = static_cast<const TQ *>(a.q) + (int64_t)(lo + t) * a.ld_q + (int64_t)h * D;
    float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      qv[e] = Elem<TQ>::load1(q + lane * E + e) * a.scale;
      o[e] = 0.f;
    }
    const int last = kv_len - len + t;
    for (int j = 0; j <= last; ++j) {
      const int id = c.table[(int64_t)slot * c.max_pages + (j >> c.page_log2)];
      if (id < 0 || id >= c.n_pages) {
        raise_error(c.err, GDN_DEVERR_PAGE);
        continue;
      }
      const int64_t blk = c.block(layer, id, hk);
      const int64_t at =
          ((blk << c.page_log2) + (j & (c.page_tokens - 1))) * D + lane * E;
      float kx[E < 4 ? 4 : E], vx[E < 4 ? 4 : E];
      if (E == 2) {
        const float4 x = kv::Code<CODE>::decode4(*reinterpret_cast<const uint16_t *>(c.k + at));
        const float4 y = kv::Code<CODE>::decode4(*reinterpret_cast<const uint16_t *>(c.v + at));
        kx[0] = x.x, kx[1] = x.y, vx[0] = y.x, vx[1] = y.y;
      } else {
#pragma unroll
        for (int e = 0; e + 3 < E; e += 4) {
          const float4 x =
              kv::Code<CODE>::decode4(*reinterpret_cast<const uint32_t *>(c.k + at + e));
          const float4 y =
              kv::Code<CODE>::decode4(*reinterpret_cast<const uint32_t *>(c.v + at + e));
          kx[e] = x.x, kx[e + 1] = x.y, kx[e + 2] = x.z, kx[e + 3] = x.w;
          vx[e] = y.x, vx[e + 1] = y.y, vx[e + 2] = y.z, vx[e + 3] = y.w;
        }
      }
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s += qv[e] * kx[e];
      s = group_sum<32>(s) * c.k_scale[blk];
      const float mn = fmaxf(m, s), keep = expf(m - mn), p = expf(s - mn);
      m = mn;
      l = l * keep + p;
      const float pv = p * c.v_scale[blk];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * keep + pv * vx[e];
    }
    TO *dst = static_cast<TO *>(a.o) + (int64_t)(lo + t) * a.ld_o + (int64_t)h * D + lane * E;
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < E; ++e) Elem<TO>::store1(dst + e, o[e] * inv);
  }
}

template <int CODE, int D, typename TQ>
cudaError_t launch_t(const KVView &c, int layer, const KVAttendArgs &a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_seqlen * c.h_q;
  int64_t bx = (rows + kWarps - 1) / kWarps;
  if (bx > 65535) bx = 65535;
  const dim3 grid((unsigned)bx, (unsigned)a.seq.n_seqs);
  if (a.o_dtype == GDN_F32)
    attend_plain_kernel<CODE, D, TQ, float><<<grid, 32 * kWarps, 0, s>>>(c, layer, a);
  else
    attend_plain_kernel<CODE, D, TQ, bf16><<<grid, 32 * kWarps, 0, s>>>(c, layer, a);
  return cudaGetLastError();
}

template <int CODE, int D>
cudaError_t by_type(const KVView &c, int layer, const KVAttendArgs &a, cudaStream_t s) {
  return a.q_dtype == GDN_F32 ? launch_t<CODE, D, float>(c, layer, a, s)
                              : launch_t<CODE, D, bf16>(c, layer, a, s);
}

template <int CODE>
cudaError_t by_dim(const KVView &c, int layer, const KVAttendArgs &a, cudaStream_t s) {
  return c.d == 64 ? by_type<CODE, 64>(c, layer, a, s)
                   : (c.d == 128 ? by_type<CODE, 128>(c, layer, a, s)
                                 : by_type<CODE, 256>(c, layer, a, s));
}

}  // namespace

cudaError_t launch_kv_attend(const KVView &c, int layer, const KVAttendArgs &a, int sm_count,
                             cudaMemPool_t work_pool, cudaStream_t s) {
  return c.code == GDN_KV_I8 ? by_dim<GDN_KV_I8>(c, layer, a, s)
                             : by_dim<GDN_KV_E4M3>(c, layer, a, s);
}

}  // namespace gdn
