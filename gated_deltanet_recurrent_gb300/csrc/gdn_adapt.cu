// The input projection with a low-rank adapter per token:
//     y[t] = W x[t] + scale[a] B[a] (A[a] x[t]),   a = ids[t]   (W x[t] alone where ids[t] = -1).
//
// gdn_adapt_low.cu has computed h[t] = scale[a] A[a] x[t]; here both products meet in one
// accumulator, so that y is rounded and written once.
//
// The tile is 128 outputs x BT tokens, the transpose of the plain projection's: W and B[a] are the
// M operand, x and h the N operand.  So few tokens make narrow tiles instead of empty rows, and the
// tokens that share an adapter (a group) are columns: its product needs only the pieces of 16
// columns that hold some of them, with zero rows in h for tokens that belong to others.  A unit is
// one group's B[a] tile of KW ranks with those rows of h, split into bf16 parts (two for a bf16 y,
// which leave 2^-16 of h, three for a float32 y, 2^-24).  The units have their own accumulator:
// products into one place run in the order of issue only if they have one shape.
//
//   warp 0      one lane: TMA of W and x tiles (a ring of k-blocks of 64) and of B tiles (a ring of
//               units)
//   warp 1      one lane: tcgen05.mma; the units are spread over the second half of the k-blocks,
//               at fixed places (the order of the sum is fixed)
//   warps 2..5  epilogue: thread = output row, from TMEM to y
//   warps 6..9  find the groups; then a warp per unit: h rows to shared memory, and a look at the B
//               tile: elements that are not finite would spoil other tokens of the range (0 * inf),
//               so they are taken out, and their products added in the epilogue to the tokens
//               that they belong to
//
// A decode step is bound by the bytes of W and of the B in use.  With fewer tiles than SMs, the CTAs
// of a cluster split the k-blocks and the units of a tile and add their parts through
// distributed shared memory, in a fixed order.  The kernel starts under the low side's (it
// waits for h only), so W is on its way early.  Every wait is bounded (GDN_DEVERR_TIMEOUT).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_adapt.h"
#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kBM = 128, kBK = 64;
constexpr int kThreads = 320;
constexpr int kBuilders = 4;  // warps
constexpr int kTileW = kBM * kBK * 2;

template <int BT, int KW, typename TO>
struct Cfg {
  static constexpr int kParts = sizeof(TO) == 4 ? 3 : 2;
  static constexpr int kStage = kTileW + BT * kBK * 2;
  static constexpr int kPitch = KW * 2;                  // bytes of a row of a unit's operands
  static constexpr int kTileB = kBM * kPitch;
  static constexpr int kTileH = BT * kPitch;             // one part
  static constexpr int kSlot = kTileB + kParts * kTileH;
  // two CTAs per SM, but for wide units and wide tiles
  static constexpr bool kTwo = BT == 16 || (BT == 64 && KW == 16);
  static constexpr int kRoom = (kTwo ? 112 : 225) * 1024 - 1024;
  static constexpr int kSlots = BT == 16 ? (KW == 16 ? 6 : 2) : kTwo ? 3 : 4 - (BT == 64);
  // warps that build units: a slot is always the same warp's, which then is never two rounds ahead
  static constexpr int kTeam = kSlots % 4 == 0 ? 4 : kSlots % 3 == 0 ? 3 : 2;
  static constexpr int kFit = (kRoom - kSlots * kSlot) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kStage + kSlots * kSlot + 1024;
  static constexpr uint32_t kTmem = 2 * BT;  // the projection's columns, then the units'
  static_assert(kStages >= 3 && kSlots % kTeam == 0, "rings");
  static_assert(BT * kBM * 4 <= kStages * kStage, "a cluster's parts take the ring's place");
};

__device__ __forceinline__ void tma_load2(void *dst, const CUtensorMap *m, int x, int y,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}

// K-major operand with rows of `pitch` bytes (32, 64 or 128) in the swizzle of that width
template <int PITCH>
__device__ __forceinline__ uint64_t operand(uint32_t saddr) {
  constexpr uint64_t kMode = PITCH == 128 ? 2 : PITCH == 64 ? 4 : 6;
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
         ((uint64_t)((8 * PITCH) >> 4) << 32) | ((uint64_t)1 << 46) | (kMode << 61);
}
// where the swizzle puts byte `off` of such a tile
template <int PITCH>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
  return off ^ (((off >> 7) & (PITCH / 16 - 1)) << 4);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void *p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float ld_peer(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int ld_peer_int(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// (try_wait may suspend the thread for a while; a producer of two rings must not)
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

// A bounded wait that also ends when the CTA gives up.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  for (uint32_t it = 0; it < (1u << 20); ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 15) == 15 && *abort_flag) return false;
  }
  return false;
}

// The groups of a tile: tokens that share an adapter.
template <int BT>
struct Groups {
  int id[BT];             // per token: its adapter, or -1
  int adapter[BT];        // per group
  unsigned short pieces[BT];  // bit p: tokens 16 p .. 16 p + 15 hold some of it
  int n;
  unsigned int bad[BT * 8 / 32];  // units (group * chunks + chunk) with elements that are not finite
  int any_bad;
};

// Run by the builder warps.  ids of tokens tok0 ..; kernels before this one wrote them.
template <int BT>
__device__ __forceinline__ void find_groups(const AdaptArgs &g, int tok0, Groups<BT> &s, int *counts) {
  const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
  if (tid < BT) {
    int id = tok0 + tid < g.tokens ? g.ids[tok0 + tid] : -1;
    if (id < 0 || id >= g.n_adapters) id = -1;
    s.id[tid] = id;
  }
  for (int i = tid; i < BT * 8 / 32; i += 128) s.bad[i] = 0;
  asm volatile("bar.sync 1, 128;" ::: "memory");
  const int id = tid < BT ? s.id[tid] : -1;
  bool lead = id >= 0;
  unsigned pieces = 0;
  if (lead) {
    for (int j = 0; j < BT; ++j) {
      if (s.id[j] != id) continue;
      if (j < tid) lead = false;
      pieces |= 1u << (j >> 4);
    }
  }
  const uint32_t m = __ballot_sync(0xffffffffu, lead);
  if (lane == 0) counts[warp] = __popc(m);
  asm volatile("bar.sync 1, 128;" ::: "memory");
  int at = __popc(m & ((1u << lane) - 1)), n = 0;
#pragma unroll
  for (int w = 0; w < kBuilders; ++w) {
    if (w < warp) at += counts[w];
    n += counts[w];
  }
  if (lead) {
    s.adapter[at] = id;
    s.pieces[at] = (unsigned short)pieces;
  }
  if (tid == 0) s.n = n, s.any_bad = 0;
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// Eight elements of h as PARTS bf16 vectors whose sum they are.
template <int PARTS>
__device__ __forceinline__ void split8(const float *h, uint4 *out) {
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = h[e];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(rest[2 * j], rest[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&b);
      const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
      // (what is infinite or NaN is the first part alone)
      rest[2 * j] = fabsf(lo) < INFINITY ? rest[2 * j] - lo : 0.f;
      rest[2 * j + 1] = fabsf(hi) < INFINITY ? rest[2 * j + 1] - hi : 0.f;
    }
    out[p] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One warp: the rows of h of a unit, columns [k0, k0 + KW), into the operand tiles at `dst`: the
// group's pieces, zeros for other tokens.
template <int BT, int KW, int PARTS>
__device__ __forceinline__ void build_rows(const AdaptArgs &g, const Groups<BT> &s, int group,
                                           int tok0, int k0, unsigned char *dst) {
  constexpr int kPer = KW / 8, kRows = 32 / kPer;  // lanes per row, rows per pass
  constexpr int kPasses = BT / kRows, kAhead = kPasses < 4 ? kPasses : 4;
  const int lane = threadIdx.x & 31, sub = lane % kPer, row = lane / kPer;
  const int id = s.adapter[group], ld = g.rank16();
  const unsigned pieces = s.pieces[group];
  const bool in = k0 + 8 * sub < ld;
  for (int p0 = 0; p0 < kPasses; p0 += kAhead) {
    float4 u[kAhead], v[kAhead];  // the loads of several passes are on their way at once
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = (p0 + i) * kRows + row;
      u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (in && s.id[r] == id) {
        const float4 *h =
            reinterpret_cast<const float4 *>(g.h + (int64_t)(tok0 + r) * ld + k0 + 8 * sub);
        u[i] = h[0], v[i] = h[1];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = (p0 + i) * kRows + row;
      if (!(pieces >> (r >> 4) & 1)) continue;
      const float e[8] = {u[i].x, u[i].y, u[i].z, u[i].w, v[i].x, v[i].y, v[i].z, v[i].w};
      uint4 part[PARTS];
      split8<PARTS>(e, part);
      const uint32_t off = swizzled<2 * KW>((uint32_t)(r * 2 * KW + sub * 16));
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        *reinterpret_cast<uint4 *>(dst + p * BT * 2 * KW + off) = part[p];
    }
  }
}

// One warp: takes infinities and NaN out of a B tile; true if there were any.
template <int BYTES>
__device__ __forceinline__ bool take_out(unsigned char *tile) {
  const int lane = threadIdx.x & 31;
  bool any = false;
#pragma unroll 4
  for (int i = lane * 16; i < BYTES; i += 512) {
    uint4 *p = reinterpret_cast<uint4 *>(tile + i);
    uint4 v = *p;
    const uint32_t a = __vcmpeq2(v.x & 0x7f807f80u, 0x7f807f80u),
                   b = __vcmpeq2(v.y & 0x7f807f80u, 0x7f807f80u),
                   c = __vcmpeq2(v.z & 0x7f807f80u, 0x7f807f80u),
                   d = __vcmpeq2(v.w & 0x7f807f80u, 0x7f807f80u);
    if (a | b | c | d) {
      any = true;
      *p = make_uint4(v.x & ~a, v.y & ~b, v.z & ~c, v.w & ~d);
    }
  }
  return __any_sync(0xffffffffu, any);
}

// The products that take_out left out, of output row n and token i of the tile.
template <int BT, int KW>
__device__ __noinline__ float put_back(const AdaptArgs &g, const Groups<BT> &s, int tok0, int i,
                                       int n) {
  float sum = 0.f;
  const int chunks = (g.rank16() + KW - 1) / KW;
  for (int gr = 0; gr < s.n; ++gr) {
    if (s.adapter[gr] != s.id[i]) continue;
    const bf16 *b = static_cast<const bf16 *>(g.b) + ((int64_t)s.id[i] * g.n_out + n) * g.ld_b;
    const float *h = g.h + (int64_t)(tok0 + i) * g.rank16();
    for (int c = 0; c < chunks; ++c) {
      const int u = gr * chunks + c;
      if (!(s.bad[u >> 5] >> (u & 31) & 1)) continue;
      for (int r = c * KW; r < min((c + 1) * KW, g.rank); ++r) {
        const float v = __bfloat162float(b[r]);
        if (!(fabsf(v) < INFINITY)) sum += v * h[r];
      }
    }
  }
  return sum;
}

template <int BT, int KW, typename TO>
__global__ void __launch_bounds__(kThreads, Cfg<BT, KW, TO>::kTwo ? 2 : 1)
    adapt_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                 const __grid_constant__ CUtensorMap mb, const __grid_constant__ AdaptArgs g,
                 int splits) {
  using C = Cfg<BT, KW, TO>;
  constexpr int S = C::kStages, E = C::kSlots, PARTS = C::kParts;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], b_full[E], x_full[E], x_empty[E], list, zeroed,
      done, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort, s_counts[kBuilders];
  __shared__ Groups<BT> s_groups;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  auto tile_w = [&](int s) { return smem + s * C::kStage; };
  auto tile_x = [&](int s) { return smem + s * C::kStage + kTileW; };
  auto slot_b = [&](int e) { return smem + S * C::kStage + e * C::kSlot; };
  auto slot_h = [&](int e) { return slot_b(e) + C::kTileB; };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part = (int)cluster_rank() % splits;
  const int n0 = (int)(blockIdx.x / splits) * kBM, tok0 = blockIdx.y * BT;
  const int blocks = (g.hidden + kBK - 1) / kBK;
  const int kb0 = (int)((int64_t)blocks * part / splits);
  const int kbs = (int)((int64_t)blocks * (part + 1) / splits) - kb0;
  const int chunks = (g.rank16() + KW - 1) / KW;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int e = 0; e < E; ++e) {
      mbar_init(&b_full[e], 1);
      mbar_init(&x_full[e], 1);
      mbar_init(&x_empty[e], 1);
    }
    mbar_init(&list, kBuilders * 32);
    mbar_init(&zeroed, 4);
    mbar_init(&done, 1);
    mbar_init(&drain, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) tc::tmem_alloc(&tmem_slot, C::kTmem);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int *abort_flag = &s_abort;
  auto fail = [&]() {
    *abort_flag = 1;
    raise_error(g.err, GDN_DEVERR_TIMEOUT);
  };
  // this CTA's units are u = part, part + splits, ... of all; the j-th of them
  auto my_units = [&]() { return (s_groups.n * chunks - part + splits - 1) / splits; };

  if (warp == 0 && lane == 0) {
    // producer: k-blocks and units as their slots get free, units as soon as the groups are known
    int kb = 0, u = 0, units = -1;
    bool good = true;
    uint32_t idle = 0;
    while (good && (kb < kbs || u < units || units < 0)) {
      bool moved = false;
      if (kb < kbs) {
        const int s = kb % S;
        if (kb < S || mbar_test_wait(&empty[s], ((kb / S) - 1) & 1)) {
          mbar_arrive_expect_tx(&full[s], C::kStage);
          tma_load2(tile_w(s), &mw, (kb0 + kb) * kBK, n0, &full[s]);
          tma_load2(tile_x(s), &mx, (kb0 + kb) * kBK, tok0, &full[s]);
          ++kb;
          moved = true;
        }
      }
      if (units < 0) {
        if (mbar_test_wait(&list, 0)) units = my_units();
      } else if (u < units) {
        const int e = u % E;
        if (u < E || mbar_test_wait(&x_empty[e], ((u / E) - 1) & 1)) {
          const int unit = part + u * splits, gr = unit / chunks, c = unit - gr * chunks;
          mbar_arrive_expect_tx(&b_full[e], C::kTileB);
          tma_load2(slot_b(e), &mb, c * KW, s_groups.adapter[gr] * g.n_out + n0, &b_full[e]);
          ++u;
          moved = true;
        }
      }
      idle = moved ? 0 : idle + 1;
      if (idle > (1u << 25)) fail();  // seconds
      if ((idle & 15) == 15) good = *abort_flag == 0;
    }
    if (!good) {  // let the copies still in flight land before the CTA exits
      for (int i = kb - S < 0 ? 0 : kb - S; i < kb; ++i)
        mbar_wait_bounded(&full[i % S], (i / S) & 1);
      for (int i = u - E < 0 ? 0 : u - E; i < u; ++i)
        mbar_wait_bounded(&b_full[i % E], (i / E) & 1);
    }
  } else if (warp == 1 && lane == 0) {
    // MMA issuer
    constexpr uint32_t kFull = tc::idesc_bf16(kBM, BT), kPiece = tc::idesc_bf16(kBM, 16);
    bool good = true;
    int u = 0, units = 0;
    const int half = kbs / 2;
    for (int kb = 0; kb < kbs && good; ++kb) {
      const int s = kb % S;
      if (!wait(&full[s], (kb / S) & 1, abort_flag)) {
        good = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t a = smem_addr(tile_w(s)), b = smem_addr(tile_x(s));
#pragma unroll
      for (int kk = 0; kk < kBK / 16; ++kk)
        tc::mma_ss_f16(tmem, operand<128>(a + 32 * kk), operand<128>(b + 32 * kk), kFull,
                       (kb | kk) ? 1u : 0u);
      tc::mma_commit(&empty[s]);
      if (kb < half) continue;
      if (kb == half) {
        if (!wait(&list, 0, abort_flag) || !wait(&zeroed, 0, abort_flag)) {
          good = false;
          break;
        }
        units = my_units();
      }
      // units up to this place: they are spread evenly over k-blocks half .. kbs - 1
      const int upto = (int)((int64_t)units * (kb - half + 1) / (kbs - half));
      for (; u < upto; ++u) {
        const int e = u % E;
        if (!wait(&b_full[e], (u / E) & 1, abort_flag) ||
            !wait(&x_full[e], (u / E) & 1, abort_flag)) {
          good = false;
          break;
        }
        tc::fence_after_sync();
        const int unit = part + u * splits, gr = unit / chunks, c = unit - gr * chunks;
        const uint32_t bt = smem_addr(slot_b(e)), ht = smem_addr(slot_h(e));
        const int steps = min(KW, g.rank16() - c * KW) / 16;
        for (unsigned m = s_groups.pieces[gr]; m != 0; m &= m - 1) {
          const int piece = __ffs(m) - 1;
          for (int p = 0; p < PARTS; ++p)
            for (int kk = 0; kk < steps; ++kk)
              tc::mma_ss_f16(tmem + BT + 16 * piece, operand<C::kPitch>(bt + 32 * kk),
                             operand<C::kPitch>(ht + p * C::kTileH + piece * 16 * C::kPitch +
                                                32 * kk),
                             kPiece, 1u);
        }
        tc::mma_commit(&x_empty[e]);
      }
    }
    if (!good) fail();
    tc::mma_commit(good ? &done : &drain);
    if (!good) mbar_wait_bounded(&drain, 0);  // MMAs in flight finish before TMEM is freed
  } else if (warp >= 6) {
    // builders
    find_groups<BT>(g, tok0, s_groups, s_counts);
    mbar_arrive(&list);
    kv::dependent_wait();  // h
    const int units = my_units();
    for (int u = warp - 6; warp - 6 < C::kTeam && u < units; u += C::kTeam) {
      const int e = u % E;
      // warp-uniform decisions
      if (!__all_sync(0xffffffffu, u < E || wait(&x_empty[e], ((u / E) - 1) & 1, abort_flag))) {
        fail();
        break;
      }
      const int unit = part + u * splits, gr = unit / chunks, c = unit - gr * chunks;
      build_rows<BT, KW, PARTS>(g, s_groups, gr, tok0, c * KW, slot_h(e));
      if (!__all_sync(0xffffffffu, wait(&b_full[e], (u / E) & 1, abort_flag))) {
        fail();
        break;
      }
      if (take_out<C::kTileB>(slot_b(e)) && lane == 0) {
        atomicOr(&s_groups.bad[unit >> 5], 1u << (unit & 31));
        s_groups.any_bad = 1;
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_full[e]);
    }
  } else if (warp >= 2) {
    // epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31, a lane per output row
    const int quad = warp & 3, row = 32 * quad + lane, n = n0 + row;
    const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16);
    {  // the units add to zeros
      const float zero[16] = {};
#pragma unroll
      for (int c = 0; c < BT / 16; ++c) tc::tmem_st16(mine + BT + 16 * c, zero);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&zeroed);
    }
    // warp-uniform decision: tcgen05.ld is a whole-warp instruction
    const bool got = __all_sync(0xffffffffu, wait(&done, 0, abort_flag));
    if (!got) {
      fail();
    } else {
      tc::fence_after_sync();
      const bool bad = s_groups.any_bad != 0;
      float *parts = reinterpret_cast<float *>(smem);  // [BT][128]: the ring is empty
      TO *y = static_cast<TO *>(g.y);
#pragma unroll 1
      for (int c = 0; c < BT / 16; ++c) {
        if (tok0 + 16 * c >= g.tokens) break;
        float v[32];
        tc::tmem_ld32(mine + 16 * c, mine + BT + 16 * c, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += v[16 + j];
        if (bad && n < g.n_out) {
          kv::dependent_wait();
          for (int j = 0; j < 16; ++j)
            if (tok0 + 16 * c + j < g.tokens)
              v[j] += put_back<BT, KW>(g, s_groups, tok0, 16 * c + j, n);
        }
        if (splits > 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) parts[(16 * c + j) * kBM + row] = v[j];
        } else if (n < g.n_out) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (tok0 + 16 * c + j < g.tokens)
              Elem<TO>::store1(y + (int64_t)(tok0 + 16 * c + j) * g.ld_y + n, v[j]);
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
  if (splits > 1) {
    // each CTA adds up its share of the tile's tokens
    __syncwarp();
    cluster_sync();
    bool sound = true;
    for (int p = 0; p < splits; ++p) sound = sound && ld_peer_int(peer_addr(&s_abort, p)) == 0;
    const int live = min(BT, g.tokens - tok0);
    const int lo = live * part / splits, hi = live * (part + 1) / splits;
    for (int i = lo * kBM + tid; sound && i < hi * kBM; i += kThreads) {
      const int t = i / kBM, n = n0 + i % kBM;
      float sum = 0.f;
      for (int p = 0; p < splits; ++p)
        sum += ld_peer(peer_addr(reinterpret_cast<float *>(smem) + i, p));
      if (n < g.n_out)
        Elem<TO>::store1(static_cast<TO *>(g.y) + (int64_t)(tok0 + t) * g.ld_y + n, sum);
    }
    cluster_sync();
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

// [rows][cols] bf16 with row stride ld elements, boxes of `box_cols` (16, 32 or 64) x box_rows in
// the swizzle of that width
bool encode_rows(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld,
                 int box_cols, int box_rows) {
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

template <int BT, int KW, typename TO>
cudaError_t launch(const AdaptArgs &g, cudaStream_t s) {
  using C = Cfg<BT, KW, TO>;
  CUtensorMap mw, mx, mb;
  if (!encode_rows(&mw, g.w, g.n_out, g.hidden, g.ld_w, kBK, kBM) ||
      !encode_rows(&mx, g.x, g.tokens, g.hidden, g.ld_x, kBK, BT) ||
      !encode_rows(&mb, g.b, (int64_t)g.n_adapters * g.n_out, g.rank, g.ld_b, KW, kBM))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> seen{0};
  const cudaError_t e = kv::allow_smem(adapt_kernel<BT, KW, TO>, C::kSmem, g.device, seen);
  if (e != cudaSuccess) return e;
  const int tiles = (g.n_out + kBM - 1) / kBM, rows = (g.tokens + BT - 1) / BT;
  const int blocks = (g.hidden + kBK - 1) / kBK;
  int splits = 1;
  while ((int64_t)tiles * rows * splits < g.sm_count && splits < 8 && blocks >= 8 * splits)
    splits *= 2;
  return kv::launch(adapt_kernel<BT, KW, TO>, dim3((unsigned)(tiles * splits), (unsigned)rows),
                    kThreads, C::kSmem, s, splits, mw, mx, mb, g, splits);
}

template <typename TO>
cudaError_t launch_t(const AdaptArgs &g, cudaStream_t s) {
  const bool narrow = g.rank <= 16;
  if (g.tokens <= 16) return narrow ? launch<16, 16, TO>(g, s) : launch<16, 64, TO>(g, s);
  if (g.tokens <= 64) return narrow ? launch<64, 16, TO>(g, s) : launch<64, 64, TO>(g, s);
  return launch<128, 16, TO>(g, s);
}

}  // namespace

size_t adapt_workspace_bytes(const AdaptArgs &g) {
  return (size_t)g.tokens * g.rank16() * sizeof(float);
}

cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t s) {
  const cudaError_t e = launch_adapt_low(g, s);
  if (e != cudaSuccess) return e;
  return g.y_dtype == GDN_F32 ? launch_t<float>(g, s) : launch_t<bf16>(g, s);
}

}  // namespace gdn
