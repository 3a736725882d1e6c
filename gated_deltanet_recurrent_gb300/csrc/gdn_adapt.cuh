// What the two projection kernels with adapters share: copies, waits, clusters, and the groups of
// tokens that have one adapter.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_adapt.h"
#include "gdn_adapt_tile.cuh"
#include "gdn_kv.cuh"
#include "gdn_mma.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace adapt {

constexpr int kBM = 128, kBK = 64;
constexpr int kTileW = kBM * kBK * 2;

// k-blocks that one accumulator of a float32 y gets: the tensor core cuts its sums off, and K = 960 so
// added is 1e-6 off, whatever hidden is.
constexpr int kChain = 15;

__device__ __forceinline__ void tma_load2(void *dst, const CUtensorMap *m, int x, int y,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store into the shared memory of CTA `rank` of the cluster, at the place of `p` in this one's.
__device__ __forceinline__ void st_peer(const void *p, int rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_addr(p)),
      "r"(rank), "f"(v)
      : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// (try_wait may suspend the thread for a while; lanes that look after a slot each must not)
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Polls of a bounded wait (of up to a microsecond or two each): what one step of any role may take grows
// with hidden.
__device__ __forceinline__ uint32_t patience(const AdaptArgs &g) {
  if (g.test_flags & (GDN_TEST_ADAPT_WAIT_TIMEOUT | GDN_TEST_ADAPT_SIDE_TIMEOUT)) return 1u << 11;
  return (1u << 20) + 64u * (uint32_t)min(g.hidden, 1 << 24);
}

// A bounded wait that also ends when the CTA gives up, which sets its limit to 0.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile uint32_t *limit) {
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15) == 0 && it >= *limit) return false;
  }
}

// The helpers, HELPERS threads from warp 2 on, do the adapters' part of mixed tiles and the epilogue.
template <int HELPERS>
__device__ __forceinline__ void helpers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(HELPERS) : "memory");
}

template <int W>
__device__ __forceinline__ void load_words(const void *p, uint32_t *out) {
  if constexpr (W == 8) {
    const uint2 v = *static_cast<const uint2 *>(p);
    out[0] = v.x, out[1] = v.y;
  } else {
    const uint4 v = *static_cast<const uint4 *>(p);
    out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
  }
}

// The groups of a mixed tile: tokens with one adapter, and the tasks, up to eight tokens of a group
// each.  Groups are in the order of their first tokens, tasks in the order of the groups.
template <int BT>
struct Groups {
  alignas(16) int id[BT];   // per token: its adapter if it is this CTA's to do, or -1
  int adapter[BT];          // per group
  short first[BT];          // of a group: its first task, and how many there are
  short count[BT];
  short start[BT];          // per token that is the first of a group: the group's first task
  short group[BT];          // per task
  unsigned char tokens[BT]; // per task: how many of the eight there are
  alignas(8) unsigned char token[BT][8];
  int sums[8];
  int n, tasks;
};

// Run by the helpers, with s.id set.
template <int BT, int HELPERS>
__device__ __forceinline__ void find_groups(Groups<BT> &s) {
  // threads that look for a token's others
  constexpr int kPer = HELPERS >= 8 * BT ? (BT >= 64 ? 8 : 4) : HELPERS >= 2 * BT ? 2 : 1;
  static_assert(HELPERS > 256 && HELPERS >= BT, "a thread per token, and one behind the last");
  const int tid = threadIdx.x - 64;
  const int token = tid / kPer, sub = tid % kPer, id = token < BT ? s.id[token < BT ? token : 0] : -1;
  int lead = BT, rank = 0, size = 0;
#pragma unroll 4
  for (int j = 4 * sub; j < BT; j += 4 * kPer) {
    const int4 other = *reinterpret_cast<const int4 *>(&s.id[j]);
    const int o[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
    for (int x = 3; x >= 0; --x)
      if (o[x] == id) {
        lead = min(lead, j + x);
        rank += j + x < token;
        ++size;
      }
  }
#pragma unroll
  for (int o = 1; o < kPer; o <<= 1) {
    lead = min(lead, __shfl_xor_sync(0xffffffffu, lead, o));
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
    size += __shfl_xor_sync(0xffffffffu, size, o);
  }
  // (for now `adapter` is the size of the group that a token is the first of)
  if (sub == 0 && token < BT) s.adapter[token] = id >= 0 && lead == token ? size : 0;
  helpers_sync<HELPERS>();
  // groups (upper half) and tasks (lower half) before each token
  const int own = tid < BT ? s.adapter[tid] : 0, tasks = (own + 7) / 8;
  const int mine = own > 0 ? (1 << 16) + tasks : 0;
  int sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if ((tid & 31) >= o) sum += y;
  }
  if ((tid & 31) == 31 && tid < 256) s.sums[tid >> 5] = sum;
  helpers_sync<HELPERS>();
  int before = sum - mine;
  for (int w = 0; w < min(tid >> 5, 8); ++w) before += s.sums[w];
  if (own > 0) {
    const int at = before >> 16, task = before & 0xffff;
    s.adapter[at] = s.id[tid];  // (at <= tid: every thread has read its place)
    s.first[at] = s.start[tid] = (short)task;
    s.count[at] = (short)tasks;
    for (int i = 0; i < tasks; ++i) {
      s.tokens[task + i] = (unsigned char)min(8, own - 8 * i);
      s.group[task + i] = (short)at;
    }
  }
  if (tid == 256) s.n = before >> 16, s.tasks = before & 0xffff;  // (all tokens are before this thread)
  helpers_sync<HELPERS>();
  if (sub == 0 && id >= 0) {
    s.token[s.start[lead] + rank / 8][rank % 8] = (unsigned char)token;
    // (the last task's empty columns have the group's first token, and are dropped)
    if (rank + 1 == size)
      for (int i = size; i & 7; ++i) s.token[s.start[lead] + i / 8][i % 8] = (unsigned char)lead;
  }
  helpers_sync<HELPERS>();
}

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      fn = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  return encode;
}

// [rows][cols] bf16 with row stride ld elements, boxes of box_cols (16, 32 or 64) x box_rows in the
// swizzle of that width
inline bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
                 int box_rows, int box_cols = kBK) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t elem[2] = {1, 1};
  const CUtensorMapSwizzle swizzle = box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_32B;
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace adapt
}  // namespace gdn
