// The input projection with a low-rank adapter per token:
//     y[t] = W x[t] + scale[a] B[a] (A[a] x[t]),   a = ids[t]   (W x[t] alone where ids[t] = -1).
//
// gdn_adapt_low.cu has computed h[t] = scale[a] A[a] x[t] and split it into bf16 parts whose sum it is
// (two for a bf16 y, which leave 2^-16 of h, three for a float32 y, 2^-24); here y is formed from both
// products and rounded and written once.
//
// The tile is 128 outputs x BT tokens, the transpose of the plain projection's: W is the M operand
// and x the N operand, so that few tokens make narrow tiles instead of empty rows.
//
//   warp 0      one lane: TMA of W and x tiles, a ring of k-blocks of 64
//   warp 1      one lane: tcgen05.mma into the tile's accumulator in TMEM
//   warps 2..9  the adapters' part of mixed tiles, then the epilogue
//
// Where all tokens of a tile have one adapter (prompts), its part is a few more k-blocks: B tiles for
// W's and the parts of h for x's.  Other tiles are mixed.  There a warp has 16 output rows and takes
// the tokens eight at a time: for each adapter among the eight, mma.sync of its 16 rows of B, straight
// from global memory to registers (several steps ahead), with the eight columns of h, of which it
// keeps those of the adapter's own tokens.  So the cost goes by tokens and hardly by adapters, and
// the work is beside the tensor core's that does W x.  The result goes to TMEM columns of its own (the
// fragment is the 16x256b shape of tcgen05.st), where the epilogue adds it.  Either way nothing of one
// request's adapter, be it infinite, meets another request's tokens.
//
// A decode step is bound by the bytes of W and of the B in use.  With fewer tiles than SMs, the CTAs
// of a cluster split the k-blocks and the tokens' eights of a tile and add their parts through
// distributed shared memory, in a fixed order.  The kernel starts under the low side's: W is on its
// way, and B asked into L2, before h is complete.  Every wait is bounded (GDN_DEVERR_TIMEOUT).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_adapt.h"
#include "gdn_kv.cuh"
#include "gdn_mma.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 320;
constexpr int kTileW = kBM * kBK * 2;

template <int BT, typename TO, bool SPLIT>
struct Cfg {
  static constexpr int kParts = sizeof(TO) == 4 ? 3 : 2;
  // The tensor core cuts its sums off: one accumulator over K = 2048 is 2e-6 off, three that take
  // the k-blocks in turn a third of that, which a bf16 y would not show.
  static constexpr int kAcc = sizeof(TO) == 4 ? 3 : 1;
  static constexpr uint32_t kTmem = (kAcc + 1) * BT;  // the adapters' columns are the last
  // two CTAs per SM where their registers (100 a thread) and columns suffice
  static constexpr bool kTwo = sizeof(TO) == 2;
  static constexpr int kStage = kTileW + BT * kBK * 2;
  static constexpr int kRecv = SPLIT ? BT * kBM * 4 : 0;  // the cluster's parts of a tile's share
  static constexpr int kFit = ((kTwo ? 111 : 223) * 1024 - 1024 - kRecv) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kStage + kRecv + 1024;
};

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

// 16 lanes x 8 columns of TMEM from an mma.sync result (its m16n8 fragment)
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const float *d) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(__float_as_uint(d[0])), "r"(__float_as_uint(d[1])), "r"(__float_as_uint(d[2])),
               "r"(__float_as_uint(d[3]))
               : "memory");
}

// A bounded wait that also ends when the CTA gives up.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  for (uint32_t it = 0; it < (1u << 20); ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15) == 15 && *abort_flag) return false;
  }
  return false;
}

// Elements r .. r + 3 of a row of B, zeros from `rank` on (what lies behind a row is not read).
__device__ __forceinline__ uint2 load4(const bf16 *row, int r, int rank) {
  if (r + 4 <= rank) return *reinterpret_cast<const uint2 *>(row + r);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (r + j < rank)
      w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[r + j] << (16 * (j & 1));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ int token_id(const AdaptArgs &g, int t) {
  const int id = t < g.tokens ? g.ids[t] : -1;
  return id >= 0 && id < g.n_adapters ? id : -1;
}

// The adapters that each eight tokens of a mixed tile have, in order; an eight without any is one
// entry too, of adapter 0 with no tokens.
struct Task {
  int64_t b;            // elements from the first adapter's B to this one's
  int h;                // elements from the h of the tile's first token to that of the eight's
  unsigned char eight;  // tokens 8 eight .. of the tile
  unsigned char mask;   // those of them that have this adapter
  unsigned char last;   // of the eight
};
template <int BT>
struct Tasks {
  alignas(16) Task task[BT + 8];  // (the steps are rounded up to a whole number of rounds)
  int count[BT / 8], n;
};

// Run by the 8 warps of the adapters' part, for the eights e = part, part + splits, ...
template <int BT>
__device__ __forceinline__ void list_tasks(const AdaptArgs &g, int tok0, int live, int part,
                                           int splits, Tasks<BT> &s) {
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  const int eights = (live + 7) / 8;
  for (int pass = 0; pass < 2; ++pass) {
    for (int e = warp; e < eights; e += 8) {
      const int id = lane < 8 ? token_id(g, tok0 + 8 * e + lane) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      const bool lead = e % splits == part && id >= 0 && __ffs(same) - 1 == lane;
      const uint32_t leads = __ballot_sync(0xffffffffu, lead);
      const int n = leads ? __popc(leads) : 1;
      if (pass == 0) {
        if (lane == 0) s.count[e] = n;
        continue;
      }
      int at = 0;
      for (int i = 0; i < e; ++i) at += s.count[i];
      const int mine = at + __popc(leads & ((1u << lane) - 1)), h = 8 * e * g.rank16();
      if (lead)
        s.task[mine] = {(int64_t)id * g.n_out * g.ld_b, h, (unsigned char)e, (unsigned char)same,
                        mine == at + n - 1};
      if (!leads && lane == 0) s.task[at] = {0, h, (unsigned char)e, 0, 1};
      if (e == eights - 1) {
        if (lane == 0) s.n = at + n;
        if (lane < 8) s.task[at + n + lane] = {0, 0, 0, 0, 0};
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
  }
}

// W bytes of a row of B from its element e on; PARTIAL: zeros from `rank` on (what lies behind a row
// is not read).
template <int W, bool PARTIAL>
__device__ __forceinline__ void load_ranks(const bf16 *p, int e, int rank, uint32_t *out) {
  if constexpr (PARTIAL) {
    const uint2 v = load4(p, e, rank);
    out[0] = v.x, out[1] = v.y;
  } else if constexpr (W == 8) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p + e);
    out[0] = v.x, out[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(p + e);
    out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
  }
}

// One warp: the adapters' part of 16 output rows (`row0` .. of the tile) of all tasks, to the TMEM
// columns at `delta`.  B rows and h columns meet in mma.sync with the rank as K; lane (r, c) of a
// fragment has rows r and r + 8 of B and column r of h, in loads of W bytes (W / 2 neighbouring
// ranks, those of W / 8 products: the order of K does not matter).  A step is NL such loads, up to
// 64 ranks of a task; the loads of D steps are in flight.  PARTIAL: any rank (W = 8); otherwise
// the rank is NL * 2 W, or with NL * 2 W = 64 also 128, and nothing is asked.
template <int BT, int W, int NL, int D, bool PARTIAL, int PARTS>
__device__ __forceinline__ void expand(const AdaptArgs &g, const Tasks<BT> &s, int n0, int row0,
                                       int tok0, uint32_t delta) {
  constexpr int kRanks = 2 * W, kWords = W / 4;  // ranks and words of a load
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int rank16 = g.rank16(), halves = NL * kRanks == 64 && rank16 > 64 ? 2 : 1;
  const int steps = s.n * halves;
  const int64_t part = (int64_t)g.tokens * rank16;
  const bf16 *lo = static_cast<const bf16 *>(g.b) + min(n0 + row0 + r, g.n_out - 1) * g.ld_b +
                   c * (W / 2),
             *hi = static_cast<const bf16 *>(g.b) + min(n0 + row0 + r + 8, g.n_out - 1) * g.ld_b +
                   c * (W / 2);
  // (columns of other tokens, or behind the last: whatever their h holds, they are dropped)
  const bf16 *h0 = static_cast<const bf16 *>(g.h) + (int64_t)(tok0 + r) * rank16 + c * (W / 2);
  uint32_t info[D];  // eight, mask, last
  uint32_t b[D][NL][2][kWords], h[D][NL][PARTS][kWords];
  // (no branch on the task: the loads of several steps are to be on their way together)
  auto load = [&](int d, int i) {
    i = min(i, steps);  // the first step behind the last is one of nothing
    const int4 raw = *reinterpret_cast<const int4 *>(&s.task[i >> (halves - 1)]);
    const int k0 = 64 * (i & (halves - 1));
    const int64_t at = (int64_t)((uint64_t)(uint32_t)raw.y << 32 | (uint32_t)raw.x);
    const bf16 *hp = h0 + raw.z + k0;
    info[d] = (uint32_t)raw.w;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      if (PARTIAL && k0 + kRanks * l >= rank16) break;
      const int e = k0 + kRanks * l;
      load_ranks<W, PARTIAL>(lo + at, e, g.rank - c * (W / 2), b[d][l][0]);
      load_ranks<W, PARTIAL>(hi + at, e, g.rank - c * (W / 2), b[d][l][1]);
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        load_ranks<W, false>(hp + p * part, kRanks * l, 0, h[d][l][p]);
    }
  };
  float out[4], acc[PARTS][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = 0.f;
#pragma unroll
  for (int p = 0; p < PARTS; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[p][e] = 0.f;
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  for (int i0 = 0; i0 < steps; i0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int i = i0 + d, half = i & (halves - 1), k0 = 64 * half;
#pragma unroll
      for (int l = 0; l < NL; ++l) {
        if (PARTIAL && k0 + kRanks * l >= rank16) break;
#pragma unroll
        for (int w = 0; w < kWords; w += 2) {
          const uint32_t a[4] = {b[d][l][0][w], b[d][l][1][w], b[d][l][0][w + 1],
                                 b[d][l][1][w + 1]};
#pragma unroll
          for (int p = 0; p < PARTS; ++p) mma16816(acc[p], a, h[d][l][p][w], h[d][l][p][w + 1]);
        }
      }
      const uint32_t mine = info[d], mask = mine >> (8 + 2 * c);
      load(d, i + D);
      if (half + 1 < halves) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = acc[0][e] + acc[1][e];
        if constexpr (PARTS == 3) v += acc[2][e];
        if (mask >> (e & 1) & 1) out[e] = v;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) acc[p][e] = 0.f;
      }
      if (mine >> 16 & 1) {
        tmem_st_16x8(delta + ((uint32_t)row0 << 16) + 8 * (mine & 255), out);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[e] = 0.f;
      }
    }
  }
}

// The adapter that all tokens of the tile have, -1 if none has any, -2 if it is mixed.  (A whole warp.)
template <int BT>
__device__ __forceinline__ int tile_adapter(const AdaptArgs &g, int tok0, int live) {
  const int lane = threadIdx.x & 31;
  const int one = token_id(g, tok0);
  bool same = true;
#pragma unroll
  for (int i = 0; i < (BT + 31) / 32; ++i)
    if (32 * i + lane < live) same = same && token_id(g, tok0 + 32 * i + lane) == one;
  return __all_sync(0xffffffffu, same) ? one : -2;
}

template <int BT, typename TO, bool SPLIT>
__global__ void __launch_bounds__(kThreads, Cfg<BT, TO, SPLIT>::kTwo ? 2 : 1)
    adapt_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                 const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mh,
                 const __grid_constant__ AdaptArgs g, int splits) {
  using C = Cfg<BT, TO, SPLIT>;
  constexpr int S = C::kStages;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], done, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;
  __shared__ float s_gone;  // SPLIT: another CTA of the cluster gave up
  __shared__ Tasks<BT> s_tasks;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  auto tile_w = [&](int s) { return smem + s * C::kStage; };
  auto tile_x = [&](int s) { return smem + s * C::kStage + kTileW; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = SPLIT ? (int)cluster_rank() : 0;
  const int n0 = (int)(blockIdx.x / splits) * kBM, tok0 = blockIdx.y * BT;
  const int live = min(BT, g.tokens - tok0);
  // this CTA's k-blocks of W x: from kb0 on
  const int all = (g.hidden + kBK - 1) / kBK;
  const int kb0 = (int)((int64_t)all * part / splits);
  const int plain = (int)((int64_t)all * (part + 1) / splits) - kb0;
  auto load_plain = [&](int kb) {
    const int s = kb % S;
    mbar_arrive_expect_tx(&full[s], C::kStage);
    tma_load2(tile_w(s), &mw, (kb0 + kb) * kBK, n0, &full[s]);
    tma_load2(tile_x(s), &mx, (kb0 + kb) * kBK, tok0, &full[s]);
  };
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    mbar_init(&drain, 1);
    s_abort = 0;
    s_gone = 0.f;
    mbar_fence_init();
    for (int kb = 0; kb < S && kb < plain; ++kb) load_plain(kb);  // nothing else is needed for these
  }
  // and, of a tile with one adapter, those of 64 ranks of a part of h each: from eb0 on
  const int one = tile_adapter<BT>(g, tok0, live);
  const int extra = one >= 0 ? (g.rank + kBK - 1) / kBK * C::kParts : 0;
  const int eb0 = extra * part / splits;
  const int kbs = plain + extra * (part + 1) / splits - eb0;
  if (warp == 1) tc::tmem_alloc(&tmem_slot, C::kTmem);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_arrive();  // (waited for before the first store to another CTA)
  }
  volatile int *abort_flag = &s_abort;
  auto fail = [&]() {
    *abort_flag = 1;
    raise_error(g.err, GDN_DEVERR_TIMEOUT);
  };

  if (warp == 0 && lane == 0) {
    // producer
    int issued = min(S, plain);
    for (int kb = issued; kb < kbs; ++kb) {
      const int s = kb % S;
      if (kb >= S && !wait(&empty[s], ((kb / S) - 1) & 1, abort_flag)) {
        fail();
        break;
      }
      if (kb < plain) {
        load_plain(kb);
      } else {
        // (rows of h behind the last token are another part's: columns that are not stored)
        const int e = eb0 + kb - plain, c = e / C::kParts, p = e % C::kParts;
        if (kb == plain) {
          kv::dependent_wait();
          asm volatile("fence.proxy.async.global;" ::: "memory");  // plain stores, read by TMA
        }
        mbar_arrive_expect_tx(&full[s], C::kStage);
        tma_load2(tile_w(s), &mb, c * kBK, one * g.n_out + n0, &full[s]);
        tma_load2(tile_x(s), &mh, c * kBK, p * g.tokens + tok0, &full[s]);
      }
      issued = kb + 1;
    }
    if (*abort_flag) {  // let the copies still in flight land before the CTA exits
      for (int kb = issued - S < 0 ? 0 : issued - S; kb < issued; ++kb)
        mbar_wait_bounded(&full[kb % S], (kb / S) & 1);
    }
  } else if (warp == 1 && lane == 0) {
    // MMA issuer
    constexpr uint32_t idesc = tc::idesc_bf16(kBM, BT);
    bool good = true;
    for (int kb = 0; kb < kbs; ++kb) {
      const int s = kb % S;
      if (!wait(&full[s], (kb / S) & 1, abort_flag)) {
        good = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t a = smem_addr(tile_w(s)), b = smem_addr(tile_x(s));
      const uint32_t acc = tmem + (uint32_t)(kb % C::kAcc) * BT;
      const int c = (eb0 + kb - plain) / C::kParts;
      const int steps = kb < plain ? kBK / 16 : min(kBK, g.rank16() - c * kBK) / 16;
#pragma unroll
      for (int kk = 0; kk < kBK / 16; ++kk)
        if (kk < steps)
          tc::mma_ss_f16(acc, tc::smem_desc_sw128(a + 32 * kk), tc::smem_desc_sw128(b + 32 * kk),
                         idesc, kb >= C::kAcc || kk > 0 ? 1u : 0u);
      tc::mma_commit(&empty[s]);
    }
    if (!good) fail();
    tc::mma_commit(good ? &done : &drain);
    if (!good) mbar_wait_bounded(&drain, 0);  // MMAs in flight finish before TMEM is freed
  } else if (warp >= 2) {
    const int quad = warp & 3, side = (warp - 2) >> 2;  // TMEM lanes 32 quad .., two warps to each
    // the adapters' part of rows 32 quad + 16 side .. + 15
    const int row0 = 32 * quad + 16 * side;
    const uint32_t delta = tmem + C::kAcc * BT;
    if (one >= 0) {  // B on its way to L2
      const bf16 *b = static_cast<const bf16 *>(g.b) +
                      ((int64_t)one * g.n_out + min(n0 + row0 + (lane & 15), g.n_out - 1)) * g.ld_b +
                      (lane >> 4) * 64;
      if ((lane >> 4) * 64 < g.rank) prefetch_l2(b);
    } else if (one == -2) {
      list_tasks<BT>(g, tok0, live, part, splits, s_tasks);
      // B on its way to L2 meanwhile
      const bf16 *mine = static_cast<const bf16 *>(g.b) +
                         min(n0 + row0 + (lane & 15), g.n_out - 1) * g.ld_b + (lane >> 4) * 64;
      for (int i = 0; i < s_tasks.n; ++i)
        if (s_tasks.task[i].mask != 0 && (lane >> 4) * 64 < g.rank)
          prefetch_l2(mine + s_tasks.task[i].b);
      kv::dependent_wait();  // h
      if (g.rank == 16)
        expand<BT, 8, 1, 6, false, C::kParts>(g, s_tasks, n0, row0, tok0, delta);
      else if (g.rank == 32)
        expand<BT, 16, 1, 4, false, C::kParts>(g, s_tasks, n0, row0, tok0, delta);
      else if (g.rank == 64 || g.rank == 128)
        expand<BT, 16, 2, 2, false, C::kParts>(g, s_tasks, n0, row0, tok0, delta);
      else
        expand<BT, 8, 4, 1, true, C::kParts>(g, s_tasks, n0, row0, tok0, delta);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    // epilogue: a lane per output row, the two warps take turns in the columns
    const int row = 32 * quad + lane, n = n0 + row;
    __syncwarp();
    if constexpr (SPLIT) cluster_wait();  // the others run
    // warp-uniform decision: tcgen05.ld is a whole-warp instruction
    const bool got = __all_sync(0xffffffffu, wait(&done, 0, abort_flag));
    if (!got) {
      fail();
    } else {
      tc::fence_after_sync();
      // SPLIT: CTA i of the cluster adds up tokens i * share ..; it receives [splits][share][128]
      float *recv = reinterpret_cast<float *>(smem + S * C::kStage);
      const int share = BT / splits;
      TO *y = static_cast<TO *>(g.y);
      const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16);
#pragma unroll 1
      for (int c = 16 * side; c < live; c += 32) {
        float v[32];
        if (one == -2) {
          tc::tmem_ld32(mine + c, mine + C::kAcc * BT + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += v[16 + j];
        } else {
          tc::tmem_ld16(mine + c, v);
        }
        if constexpr (C::kAcc == 3) {
          float u[32];
          if (kbs > 2) {
            tc::tmem_ld32(mine + BT + c, mine + 2 * BT + c, u);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += u[j] + u[16 + j];
          } else if (kbs > 1) {
            tc::tmem_ld16(mine + BT + c, u);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += u[j];
          }
        }
        if constexpr (SPLIT) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < live)
              st_peer(recv + (part * share + (c + j) % share) * kBM + row, (c + j) / share, v[j]);
        } else if (n < g.n_out) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < live)
              Elem<TO>::store1(y + (int64_t)(tok0 + c + j) * g.ld_y + n, v[j]);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmem);
  }
  if constexpr (SPLIT) {
    __syncwarp();
    if (warp < 2) cluster_wait();
    if (*abort_flag)
      for (int p = 0; p < splits; ++p) st_peer(&s_gone, p, 1.f);
    cluster_arrive();
    cluster_wait();
    const float *recv = reinterpret_cast<const float *>(smem + S * C::kStage);
    const int share = BT / splits, mine = min(share, live - part * share);
    for (int i = tid; s_gone == 0.f && i < mine * kBM; i += kThreads) {
      const int t = i / kBM, n = n0 + i % kBM;
      float sum = 0.f;
      for (int p = 0; p < splits; ++p) sum += recv[p * share * kBM + i];
      if (n < g.n_out)
        Elem<TO>::store1(
            static_cast<TO *>(g.y) + (int64_t)(tok0 + part * share + t) * g.ld_y + n, sum);
    }
  }
  // what follows on the stream waits for this kernel only: the low side is complete too
  kv::dependent_wait();
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
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

// [rows][cols] bf16 with row stride ld elements, box {64, box_rows}, 128-byte swizzle
bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
                 int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  cuuint32_t elem[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int BT, typename TO, bool SPLIT>
cudaError_t launch(const AdaptArgs &g, int splits, cudaStream_t s) {
  using C = Cfg<BT, TO, SPLIT>;
  CUtensorMap mw, mx, mb, mh;
  if (!encode_rows(&mw, g.w, g.n_out, g.hidden, g.ld_w, kBM) ||
      !encode_rows(&mx, g.x, g.tokens, g.hidden, g.ld_x, BT) ||
      !encode_rows(&mb, g.b, (int64_t)g.n_adapters * g.n_out, g.rank, g.ld_b, kBM) ||
      !encode_rows(&mh, g.h, (int64_t)C::kParts * g.tokens, g.rank16(), g.rank16(), BT))
    return cudaErrorNotSupported;
  static std::atomic<uint64_t> seen{0};
  const cudaError_t e = kv::allow_smem(adapt_kernel<BT, TO, SPLIT>, C::kSmem, g.device, seen);
  if (e != cudaSuccess) return e;
  const int tiles = (g.n_out + kBM - 1) / kBM, rows = (g.tokens + BT - 1) / BT;
  return kv::launch(adapt_kernel<BT, TO, SPLIT>, dim3((unsigned)(tiles * splits), (unsigned)rows),
                    kThreads, C::kSmem, s, splits, mw, mx, mb, mh, g, splits);
}

template <int BT, typename TO>
cudaError_t launch_bt(const AdaptArgs &g, cudaStream_t s) {
  const int64_t tiles = (int64_t)((g.n_out + kBM - 1) / kBM) * ((g.tokens + BT - 1) / BT);
  const int blocks = (g.hidden + kBK - 1) / kBK;
  // CTAs that share a tile: so many that every multiprocessor has one, with four k-blocks each at
  // least (one token, 2048 -> 12352: 194 CTAs 15 us, 97 CTAs 17; 64 tokens with an adapter each of
  // rank 64: 61 and 79)
  int splits = 1;
  while (splits * tiles < g.sm_count && splits < 8 && blocks >= 8 * splits) splits *= 2;
  return splits > 1 ? launch<BT, TO, true>(g, splits, s) : launch<BT, TO, false>(g, 1, s);
}

template <typename TO>
cudaError_t launch_t(const AdaptArgs &g, cudaStream_t s) {
  if (g.tokens <= 16) return launch_bt<16, TO>(g, s);
  // tiles of 128 tokens read W half as often, if there is one for every multiprocessor
  const int64_t wide = (int64_t)((g.n_out + kBM - 1) / kBM) * ((g.tokens + 127) / 128);
  if (g.tokens <= 64 || wide < g.sm_count) return launch_bt<64, TO>(g, s);
  return launch<128, TO, false>(g, 1, s);
}

}  // namespace

size_t adapt_workspace_bytes(const AdaptArgs &g) {
  // (eight rows more: the tokens are read by eights)
  return ((size_t)g.tokens * g.parts() + 8) * g.rank16() * 2;
}

cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t s) {
  const cudaError_t e = launch_adapt_low(g, s);
  if (e != cudaSuccess) return e;
  return g.y_dtype == GDN_F32 ? launch_t<float>(g, s) : launch_t<bf16>(g, s);
}

}  // namespace gdn
