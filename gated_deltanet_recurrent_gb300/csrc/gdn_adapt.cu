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
//   warps 2..17 the adapters' part of mixed tiles, then the epilogue
//   warp 18     a lane per slot: copies of the B tiles of a mixed tile
//
// Where all tokens of a tile have one adapter (prompts), its part is a few more k-blocks: B tiles for
// W's and the parts of h for x's.  Other tiles are mixed.  There the B tile of every adapter that the
// tile has comes through a ring of its own, by TMA too: a decode step is bound by the bytes of W and of
// the B in use, and only copies that need no registers keep enough of both on their way.  Four warps
// with 32 output rows each take an adapter's rows of B into registers, once, and multiply them by the
// h of the adapter's own tokens, eight at a time, wherever they are in the tile (mma.sync, with the
// rank as K); four such teams take the adapters in turn.  So B is read once per tile and adapter, the
// tensor core's work on W x goes on beside it, and nothing of one request's adapter, be it infinite,
// meets another request's tokens.  The results go to shared memory, [token][row], where the epilogue
// adds them.
//
// With fewer tiles than SMs, the CTAs of a cluster split the k-blocks and the adapters of a tile and
// push their parts into each other's shared memory, where they are added in a fixed order.  The
// kernel starts under the low side's: W and B are on their way before h is complete.  Every wait is
// bounded (GDN_DEVERR_TIMEOUT).
//
// Measured with the low side: one token, 2048 -> 5120, rank 16, 10.9 us (latency; its bytes take 3.1);
// 64 tokens with an adapter each, 2048 -> 12352, rank 16, 20.9 us on warm and 22.1 on cold weights (82 MB:
// 12.1), rank 64 39.9 (25.1), without adapters 18.0 (7.7).  Narrower tiles, one for each SM, take as long.
#include "gdn_adapt.cuh"

namespace gdn {
namespace {

using namespace adapt;

constexpr int kHelpers = 512;            // threads: warps 2 .. 17
constexpr int kThreads = 64 + kHelpers + 32;
constexpr int kTeams = 4;                // of four warps
constexpr int kPitch = kBM + 4;      // floats of a token's row of the adapters' part
constexpr int kRingB = 64 * 1024;    // bytes of the ring of B tiles

// The sums of one output: column at (+ BT, + 2 BT ...) of the first `used` of ACC accumulators.
template <int BT, int ACC>
__device__ __forceinline__ void add_accumulators(uint32_t at, int used, float *v) {
  tc::tmem_ld16(at, v);
#pragma unroll
  for (int a = 1; a < ACC; a += 2) {
    float u[32];
    if (a + 1 < ACC && a + 1 < used) {
      tc::tmem_ld32(at + a * BT, at + (a + 1) * BT, u);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += u[j] + u[16 + j];
    } else if (a < used) {
      tc::tmem_ld16(at + a * BT, u);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += u[j];
    }
  }
}

constexpr uint32_t pow2_at_least(uint32_t n) {
  uint32_t p = 32;
  while (p < n) p *= 2;
  return p;
}

template <int BT, int PITCH, typename TO>
struct Cfg {
  static constexpr int kParts = sizeof(TO) == 4 ? 3 : 2;
  // The tensor core cuts its sums off: one accumulator over K = 2048 is 2e-6 off, and several that
  // take the k-blocks in turn that much less each.  A bf16 y has four, so that its roundings are nearly
  // always those of the exact sum; a float32 y has as many as there is room for, and where one would get
  // more than kChain k-blocks they are taken out before (`delta`) and start anew.
  static constexpr bool kLong = sizeof(TO) == 4;
  static constexpr int kAcc = !kLong ? 4 : BT == 96 ? 5 : 8;
  static constexpr int kRound = kAcc * kChain;
  static constexpr uint32_t kTmem = pow2_at_least(kAcc * BT);
  static constexpr int kStage = kTileW + BT * kBK * 2;
  static constexpr int kDelta = BT * kPitch * 4;
  static constexpr int kH = kParts * BT * PITCH;  // h of the tile, PITCH / 2 ranks of it
  static constexpr int kFit = (224 * 1024 - kRingB - kDelta - kH) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmem = kStages * kStage + kRingB + kDelta + kH + 1024;
  static_assert(BT * kBM * 4 <= kRingB, "a cluster's parts take the place of the B tiles");
};

// A ring of B tiles of 128 rows of PITCH bytes, in the swizzle of that width.
struct RingB {
  unsigned char *tiles;
  uint64_t *full, *empty;
};
template <int PITCH>
constexpr int kSlots = kRingB / (kBM * PITCH);

// where that puts byte `off` of a tile
template <int PITCH>
__device__ __forceinline__ uint32_t swizzled(uint32_t off) {
  return off ^ (((off >> 7) & (PITCH / 16 - 1)) << 4);
}

// Where 16 bytes of h lie in shared memory, [part][token][PITCH]: two neighbouring tokens' rows take
// different banks.
template <int PITCH>
__device__ __forceinline__ int h_offset(int token, int byte) {
  return token * PITCH + (PITCH == 128 ? byte ^ ((token & 1) << 6) : byte);
}

// Run by the helpers (`warp` of them): all groups of the tile.  Unit u = half * n + group is PITCH / 2
// ranks of a group's B; it is team u % 4's, in which a warp takes 32 of its rows, as two fragments.
// Lane (r, c) of a fragment has rows r and r + 8 of B and token r of a task, for each W bytes the same
// ranks (W / 2 neighbours: the order of K does not matter).  False: a wait gave up.
template <int BT, int PITCH, int PARTS>
__device__ __forceinline__ bool expand(const AdaptArgs &g, const Groups<BT> &s, const RingB &ring,
                                       int warp, int tok0, int live, unsigned char *hs, float *delta,
                                       volatile uint32_t *limit) {
  constexpr int W = PITCH == 32 ? 8 : 16, NL = PITCH / (4 * W), kWords = W / 4;
  constexpr int E = kSlots<PITCH>;
  static_assert(E % kTeams == 0, "a slot is always the same team's, which then is never two rounds ahead");
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, row0 = 32 * (warp & 3);
  const int team = warp >> 2, ld = g.rank_pad(), halves = ld * 2 / PITCH;
  float *const to = delta + row0 + r;
  bool good = true;
  for (int half = 0; half < halves; ++half) {
    if (half > 0) helpers_sync<kHelpers>();  // the first half has been read
    // h of the tokens that have an adapter here (nothing else of it is defined, nor read)
    for (int i = 32 * warp + lane; i < PARTS * live * (PITCH / 16); i += kHelpers) {
      const int q = i / (live * (PITCH / 16)), rest = i % (live * (PITCH / 16));
      const int t = rest / (PITCH / 16), at = rest % (PITCH / 16) * 16;
      if (s.id[t] < 0) continue;
      *reinterpret_cast<uint4 *>(hs + q * (BT * PITCH) + h_offset<PITCH>(t, at)) =
          *reinterpret_cast<const uint4 *>(
              static_cast<const unsigned char *>(g.h) +
              (((int64_t)q * g.tokens + tok0 + t) * ld * 2 + half * PITCH + at));
    }
    helpers_sync<kHelpers>();
    // (units of both halves go round the teams and slots in one order)
    for (int u = half * s.n + ((team - half * s.n) & (kTeams - 1)); good && u < (half + 1) * s.n;
         u += kTeams) {
      const int group = u - half * s.n, e = u % E;
      if (!__all_sync(0xffffffffu, wait(&ring.full[e], (u / E) & 1, limit))) {
        good = false;
        break;
      }
      const unsigned char *tile = ring.tiles + e * (kBM * PITCH);
      uint32_t b[2][NL][2][kWords];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int l = 0; l < NL; ++l)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            load_words<W>(tile + swizzled<PITCH>((uint32_t)((row0 + 16 * m + r + 8 * y) * PITCH +
                                                            l * 4 * W + c * W)),
                          b[m][l][y]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[e]);
      const int first = s.first[group], end = first + s.count[group];
      for (int t = first; t < end; ++t) {
        const int col = s.token[t][r], live_cols = s.tokens[t];
        const uint32_t two = *reinterpret_cast<const unsigned short *>(&s.token[t][2 * c]);
        float acc[2][PARTS][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[m][q][x] = 0.f;
#pragma unroll
        for (int l = 0; l < NL; ++l) {
          uint32_t h[PARTS][kWords];
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            load_words<W>(hs + q * (BT * PITCH) + h_offset<PITCH>(col, l * 4 * W + c * W), h[q]);
#pragma unroll
          for (int w = 0; w < kWords; w += 2)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t a[4] = {b[m][l][0][w], b[m][l][1][w], b[m][l][0][w + 1],
                                     b[m][l][1][w + 1]};
#pragma unroll
              for (int q = 0; q < PARTS; ++q) mma16816(acc[m][q], a, h[q][w], h[q][w + 1]);
            }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {  // columns 2 c and 2 c + 1
          if (2 * c + y >= live_cols) continue;
          float *at = to + (two >> (8 * y) & 255) * kPitch;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // rows r and r + 8
              float v = acc[m][0][2 * x + y] + acc[m][1][2 * x + y];
              if constexpr (PARTS == 3) v += acc[m][2][2 * x + y];
              if (half > 0) v += at[16 * m + 8 * x];
              at[16 * m + 8 * x] = v;
            }
        }
      }
    }
  }
  return good;
}

template <int BT, int PITCH, typename TO, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    adapt_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                 const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mu,
                 const __grid_constant__ CUtensorMap mh, const __grid_constant__ AdaptArgs g,
                 int splits) {
  using C = Cfg<BT, PITCH, TO>;
  constexpr int S = C::kStages, E = kSlots<PITCH>;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], b_full[E], b_empty[E], list, done, taken,
      drain;
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t s_limit;  // of the waits
  __shared__ int s_issued, s_issued_b[E];  // k-blocks and B tiles whose copies were started
  __shared__ float s_gone;  // SPLIT: another CTA of the cluster gave up
  __shared__ Groups<BT> s_groups;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  auto tile_w = [&](int s) { return smem + s * C::kStage; };
  auto tile_x = [&](int s) { return smem + s * C::kStage + kTileW; };
  unsigned char *ring_b = smem + S * C::kStage;
  unsigned char *hs = ring_b + kRingB;
  float *delta = reinterpret_cast<float *>(hs + C::kH);  // [token][kPitch]

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
    for (int e = 0; e < E; ++e) {
      mbar_init(&b_full[e], 1);
      mbar_init(&b_empty[e], 4);
    }
    mbar_init(&list, 1);
    mbar_init(&done, 1);
    mbar_init(&taken, kHelpers / 32);
    mbar_init(&drain, 1);
    s_limit = patience(g);
    for (int e = 0; e < E; ++e) s_issued_b[e] = 0;
    s_gone = 0.f;
    mbar_fence_init();
    // (test hooks: a barrier of one CTA waits for 16 bytes that no one sends)
    if (g.test_flags != 0 && (blockIdx.x / splits + blockIdx.y) & 1 && part == splits - 1) {
      if (g.test_flags & GDN_TEST_ADAPT_WAIT_TIMEOUT) mbar_expect_tx(&full[0], 16);
      if (g.test_flags & GDN_TEST_ADAPT_SIDE_TIMEOUT) mbar_expect_tx(&b_full[0], 16);
    }
    for (int kb = 0; kb < S && kb < plain; ++kb) load_plain(kb);  // nothing else is needed for these
  }
  // the adapter that all tokens of the tile have, -1 if none has any, -2 if it is mixed (adapters i
  // with i % splits == part are then this CTA's)
  bool same = true;
  int one = token_id(g, tok0);
  if (tid < live) {
    const int id = token_id(g, tok0 + tid);
    same = id == one;
    s_groups.id[tid] = id >= 0 && id % splits == part ? id : -1;
  } else if (tid < BT) {
    s_groups.id[tid] = -1;
  }
  __syncwarp();
  if (warp == 1) tc::tmem_alloc(&tmem_slot, C::kTmem);
  tc::fence_before_sync();
  if (!__syncthreads_and(same)) one = -2;
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  // the k-blocks of a tile with one adapter: 64 ranks of a part of h each, from eb0 on
  const int extra = one >= 0 ? (g.rank + kBK - 1) / kBK * C::kParts : 0;
  const int eb0 = extra * part / splits;
  const int kbs = plain + extra * (part + 1) / splits - eb0;
  // k-blocks before the last round of the accumulators, and in it
  const int rounds_before = C::kLong ? (kbs - 1) / C::kRound : 0, last = kbs - rounds_before * C::kRound;
  const int halves = g.rank_pad() * 2 / PITCH;
  volatile uint32_t *limit = &s_limit;
  const RingB ring{ring_b, b_full, b_empty};
  auto fail = [&]() {
    *limit = 0;
    raise_error(g.err, GDN_DEVERR_TIMEOUT);
  };

  if (warp == 0 && lane == 0) {
    // producer
    int issued = min(S, plain);
    for (int kb = issued; kb < kbs; ++kb) {
      const int s = kb % S;
      if (kb >= S && !wait(&empty[s], ((kb / S) - 1) & 1, limit)) {
        fail();
        break;
      }
      if (kb < plain) {
        load_plain(kb);
      } else {
        // (rows of h behind the last token are another part's: columns that are not stored)
        const int e = eb0 + kb - plain, c = e / C::kParts, p = e % C::kParts;
        mbar_arrive_expect_tx(&full[s], C::kStage);
        tma_load2(tile_w(s), &mb, c * kBK, one * g.n_out + n0, &full[s]);
        if (kb == plain) {
          kv::dependent_wait();
          asm volatile("fence.proxy.async.global;" ::: "memory");  // plain stores, read by TMA
        }
        tma_load2(tile_x(s), &mh, c * kBK, p * g.tokens + tok0, &full[s]);
      }
      issued = kb + 1;
    }
    s_issued = issued;
  } else if (warp == 2 + kHelpers / 32) {
    // a lane per slot of the ring of B tiles
    if (one == -2) {
      bool good = __all_sync(0xffffffffu, wait(&list, 0, limit));
      const int units = good ? s_groups.n * halves : 0;
      int u = lane < E ? lane : units;
      uint32_t idle = 0;
      while (good && __any_sync(0xffffffffu, u < units)) {
        bool moved = false;
        if (u < units && (u < E || mbar_test_wait(&b_empty[lane], ((u / E) - 1) & 1))) {
          const int half = u >= s_groups.n, group = u - half * s_groups.n;
          const int row = s_groups.adapter[group] * g.n_out + n0;
          unsigned char *tile = ring_b + lane * (kBM * PITCH);
          mbar_arrive_expect_tx(&b_full[lane], kBM * PITCH);
          tma_load2(tile, &mu, half * (PITCH / 2), row, &b_full[lane]);
          u += E;
          moved = true;
        }
        idle = __any_sync(0xffffffffu, moved) ? 0 : idle + 1;
        if (idle > (1u << 24)) fail();  // seconds
        if ((idle & 15) == 15) good = !__any_sync(0xffffffffu, *limit == 0);
      }
      if (lane < E) s_issued_b[lane] = u / E;
    }
  } else if (warp == 1 && lane == 0) {
    // MMA issuer
    constexpr uint32_t idesc = tc::idesc_bf16(kBM, BT);
    bool good = true;
    int in = 0, round = 0;  // k-blocks of the round
    for (int kb = 0; kb < kbs; ++kb, ++in) {
      if (C::kLong && in == C::kRound) {
        tc::mma_commit(&done);
        good = wait(&taken, round & 1, limit);
        tc::fence_after_sync();
        in = 0, ++round;
      }
      const int s = kb % S;
      if (!good || !wait(&full[s], (kb / S) & 1, limit)) {
        good = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t a = smem_addr(tile_w(s)), b = smem_addr(tile_x(s));
      const uint32_t acc = tmem + (uint32_t)(in % C::kAcc) * BT;
      const int c = (eb0 + kb - plain) / C::kParts;
      const int steps = kb < plain ? kBK / 16 : min(kBK, g.rank16() - c * kBK) / 16;
#pragma unroll
      for (int kk = 0; kk < kBK / 16; ++kk)
        if (kk < steps)
          tc::mma_ss_f16(acc, tc::smem_desc_sw128(a + 32 * kk), tc::smem_desc_sw128(b + 32 * kk),
                         idesc, in >= C::kAcc || kk > 0 ? 1u : 0u);
      tc::mma_commit(&empty[s]);
    }
    if (good)
      tc::mma_commit(&done);
    else
      fail();
  } else if (warp >= 2) {
    bool whole = true;  // nothing was given up
    if (one >= 0) {  // B on its way to L2
      const bf16 *b = static_cast<const bf16 *>(g.b) +
                      ((int64_t)one * g.n_out + min(n0 + (tid - 64) / 4, g.n_out - 1)) * g.ld_b +
                      (tid & 3) * 64;
      if ((tid & 3) * 64 < g.rank) prefetch_l2(b);
    } else if (one == -2) {
      find_groups<BT, kHelpers>(s_groups);
      if (tid == 64) mbar_arrive(&list);
      for (int t = warp - 2; t < live; t += kHelpers / 32)  // tokens that get nothing from this CTA
        if (s_groups.id[t] < 0)
          reinterpret_cast<float4 *>(delta + t * kPitch)[lane] = make_float4(0.f, 0.f, 0.f, 0.f);
      kv::dependent_wait();  // h
      if (!expand<BT, PITCH, C::kParts>(g, s_groups, ring, warp - 2, tok0, live, hs, delta,
                                        limit))
        fail();
      helpers_sync<kHelpers>();
      whole = *limit != 0;
    }
    // a lane per output row, the four warps of TMEM lanes 32 quad .. take turns in the columns
    const int quad = warp & 3, side = (warp - 2) >> 2, row = 32 * quad + lane, n = n0 + row;
    const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16);
    // the accumulators of a long sum, taken out
    for (int r = 0; C::kLong && whole && r < rounds_before; ++r) {
      whole = __all_sync(0xffffffffu, wait(&done, r & 1, limit));
      if (!whole) {
        fail();
        break;
      }
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 16 * side; c < live; c += 64) {
        float v[16];
        add_accumulators<BT, C::kAcc>(mine + c, C::kAcc, v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < live) {
            float *at = &delta[(c + j) * kPitch + row];
            *at = one == -2 || r > 0 ? *at + v[j] : v[j];
          }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&taken);
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_arrive();  // the B tiles' place may be written by the others
      cluster_wait();
    }
    // warp-uniform decision: tcgen05.ld is a whole-warp instruction
    const bool got =
        __all_sync(0xffffffffu, whole && wait(&done, rounds_before & 1, limit));
    if (!got) {
      fail();
    } else {
      tc::fence_after_sync();
      // SPLIT: CTA i of the cluster adds up tokens i * share ..; it receives [splits][share][128]
      float *recv = reinterpret_cast<float *>(ring_b);
      const int share = (BT + splits - 1) / splits;
      TO *y = static_cast<TO *>(g.y);
#pragma unroll 1
      for (int c = 16 * side; c < live; c += 64) {
        float v[16];
        add_accumulators<BT, C::kAcc>(mine + c, last, v);
        if (one == -2 || rounds_before > 0) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < live) v[j] += delta[(c + j) * kPitch + row];
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
  if constexpr (SPLIT) {
    __syncwarp();
    if (warp < 2 || warp >= 2 + kHelpers / 32) cluster_arrive();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (*limit == 0) {  // copies and products still in flight end before the CTA does
    if (tid == 0)
      for (int kb = max(0, s_issued - S); kb < s_issued; ++kb)
        mbar_wait_bounded(&full[kb % S], (kb / S) & 1, patience(g));
    if (tid == 32) {
      tc::mma_commit(&drain);
      mbar_wait_bounded(&drain, 0, patience(g));
    }
    if (warp == 2 + kHelpers / 32 && lane < E && s_issued_b[lane] > 0)
      mbar_wait_bounded(&b_full[lane], (s_issued_b[lane] - 1) & 1, patience(g));
    __syncthreads();
  }
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmem);
  }
  if constexpr (SPLIT) {
    __syncwarp();
    if (warp < 2 || warp >= 2 + kHelpers / 32) cluster_wait();
    if (*limit == 0)
      for (int p = 0; p < splits; ++p) st_peer(&s_gone, p, 1.f);
    cluster_arrive();
    cluster_wait();
    const float *recv = reinterpret_cast<const float *>(ring_b);
    const int share = (BT + splits - 1) / splits, mine = min(share, live - part * share);
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

template <int BT, int PITCH, typename TO, bool SPLIT>
cudaError_t launch(const AdaptArgs &g, int splits, cudaStream_t s) {
  using C = Cfg<BT, PITCH, TO>;
  CUtensorMap mw, mx, mb, mu, mh;
  const int64_t rows_b = (int64_t)g.n_adapters * g.n_out, ld = g.rank_pad();
  if (!encode_rows(&mw, g.w, g.n_out, g.hidden, g.ld_w, kBM) ||
      !encode_rows(&mx, g.x, g.tokens, g.hidden, g.ld_x, BT) ||
      !encode_rows(&mb, g.b, rows_b, g.rank, g.ld_b, kBM) ||
      !encode_rows(&mu, g.b, rows_b, g.rank, g.ld_b, kBM, PITCH / 2) ||
      !encode_rows(&mh, g.h, (int64_t)C::kParts * g.tokens, ld, ld, BT))
    return cudaErrorNotSupported;
  static std::atomic<uint64_t> seen{0};
  const cudaError_t e =
      kv::allow_smem(adapt_kernel<BT, PITCH, TO, SPLIT>, C::kSmem, g.device, seen);
  if (e != cudaSuccess) return e;
  const int tiles = (g.n_out + kBM - 1) / kBM, rows = (g.tokens + BT - 1) / BT;
  return kv::launch(adapt_kernel<BT, PITCH, TO, SPLIT>,
                    dim3((unsigned)(tiles * splits), (unsigned)rows), kThreads, C::kSmem, s, splits,
                    mw, mx, mb, mu, mh, g, splits);
}

int64_t tiles_of(const AdaptArgs &g, int bt) {
  return (int64_t)((g.n_out + kBM - 1) / kBM) * ((g.tokens + bt - 1) / bt);
}

// How often tiles of bt tokens fill the device.
int64_t rounds_of(const AdaptArgs &g, int bt) {
  return (tiles_of(g, bt) + g.sm_count - 1) / g.sm_count;
}

// Tiles of 96 tokens where they take fewer rounds than tiles of 64: 256 tokens with 64 adapters of rank
// 16, 2048 -> 5120: 25.6 and 41.3 us, 96 tokens, 2048 -> 12352: 23.4 and 36.5; 192 tokens, 2048 -> 5120, in
// one round either way: 64 is faster.
bool wide_tiles(const AdaptArgs &g) {
  return rounds_of(g, 96) < rounds_of(g, 64);
}

// CTAs that share a tile: as many as fit on the device at once, with four k-blocks each at least, and
// four at most (one token, 2048 -> 5120: one CTA a tile 16.6 us, two 13.0, three 11.6; 64 tokens with an
// adapter each, 2048 -> 2048: two 17.1 us, four 13.8, eight 21.6)
int splits_of(const AdaptArgs &g, int bt) {
  const int64_t fit = g.sm_count / tiles_of(g, bt), blocks = (g.hidden + kBK - 1) / kBK;
  const int64_t most = fit < blocks / 4 ? fit : blocks / 4;
  return most < 1 ? 1 : most > 4 ? 4 : (int)most;
}

// The tile's tokens.
int tokens_of_tile(const AdaptArgs &g) {
  return g.tokens <= 16 ? 16 : wide_tiles(g) ? 96 : 64;
}

template <int BT, int PITCH, typename TO>
cudaError_t launch_split(const AdaptArgs &g, cudaStream_t s) {
  if constexpr (BT == 96) return launch<BT, PITCH, TO, false>(g, 1, s);  // (too many tiles to share any)
  const int splits = splits_of(g, BT);
  return splits > 1 ? launch<BT, PITCH, TO, true>(g, splits, s)
                    : launch<BT, PITCH, TO, false>(g, 1, s);
}

template <int BT, typename TO>
cudaError_t launch_bt(const AdaptArgs &g, cudaStream_t s) {
  return g.rank <= 16   ? launch_split<BT, 32, TO>(g, s)
         : g.rank <= 32 ? launch_split<BT, 64, TO>(g, s)
                        : launch_split<BT, 128, TO>(g, s);
}

// These kernels take calls of one tile's tokens, and others that fill the device at most twice;
// pairs of CTAs take what is longer.  With 64 adapters of rank 64 in any order and with none (us, here
// and pairs): 384 tokens, 2048 -> 5120: 65 and 104, 34 and 31; 256, 2048 -> 12352: 73 and 105, 38 and 33;
// three rounds, 384, 2048 -> 12352: 107 and 160, 57 and 37, 777 float32 tokens in runs of 50, 2048 -> 5120:
// 75 and 46.  (Up to 2048 tokens: the low side's windows are made for few.)
constexpr int kOneTile = 64, kMostTokens = 2048, kRounds = 2;

template <typename TO>
cudaError_t launch_t(const AdaptArgs &g, cudaStream_t s) {
  const int bt = tokens_of_tile(g);
  return bt == 16 ? launch_bt<16, TO>(g, s) : bt == 96 ? launch_bt<96, TO>(g, s) : launch_bt<64, TO>(g, s);
}

}  // namespace

size_t adapt_workspace_bytes(const AdaptArgs &g) {
  return (size_t)g.tokens * g.parts() * g.rank_pad() * 2 * (g.tile > 0 ? kPlanes : 1);
}

int adapt_tile(const AdaptArgs &g) {
  const bool few = g.tokens <= kOneTile ||
                   (g.tokens <= kMostTokens && rounds_of(g, tokens_of_tile(g)) <= kRounds);
  return few ? 0 : g.y_dtype == GDN_F32 ? 128 : 256;
}

cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t s) {
  // (CTAs that share a tile have so little of W each that h is what they wait for: 64 tokens with an adapter
  // each, 2048 -> 5120, 19.0 us without regard to them and 20.8 with)
  const int bt = tokens_of_tile(g);
  const int64_t tiles = tiles_of(g, bt) < g.sm_count ? tiles_of(g, bt) : g.sm_count;
  const cudaError_t e = launch_adapt_low(g, splits_of(g, bt) > 1 ? 0 : (int)tiles, s);
  if (e != cudaSuccess) return e;
  if (g.tile > 0) return launch_adapt_pair(g, s);
  return g.y_dtype == GDN_F32 ? launch_t<float>(g, s) : launch_t<bf16>(g, s);
}

}  // namespace gdn
