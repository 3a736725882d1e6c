// The projection with adapters for many tokens (see gdn_adapt.cu for the mathematics and for calls of
// few): pairs of CTAs on the 5th-generation tensor cores, tcgen05.mma cta_group::2.
//
// A pair's tile is 256 outputs x BT tokens.  Each CTA holds 128 rows of W and half of the tokens of x,
// and both halves of the products: 32 KiB of operands per k-block and CTA for 256 x 256 x 64, two thirds
// of what a CTA alone needs for as much work, so that a ring of six covers the copies' latency.  The
// pairs walk the tiles, output blocks fastest (W stays in L2).
//
//   warp 0      one lane: TMA into this CTA's ring, reported to CTA 0's barriers
//   warp 1      one lane of CTA 0: tcgen05.mma for both, commits to both
//   warps 2..13 the adapters' part of mixed tiles, then the epilogue
//   warp 14     looks a few tiles ahead: which have one adapter, or none
//
// The adapters are further k-blocks: B tiles for W's and the parts of h for x's.  Where all tokens of a
// tile have one adapter (most of a prompt) that is all.  In a mixed tile every adapter has its own
// k-blocks, with a plane of h that has zeros for the other tokens.  A result that is not finite may then
// come from another request's adapter (0 * inf), and is computed again from its own, so that nothing of
// one adapter reaches another's tokens: after a warp's last tile, 32 outputs of 16 tokens at a time, by
// mma.sync.  (Where every result of every tile is: 5000 bf16 tokens, eight adapters of rank 32, 2048 -> 1296,
// 110 -> 633 us; 600 tokens -> 40960 161 -> 2180; these are loads of W from L2, once per 16 tokens.)  For more than eight adapters in a tile
// the helpers multiply B and h with mma.sync: four warps with 32 output rows each take the tasks
// (up to eight tokens of one adapter) in turn, with B and h from global memory, and store them to TMEM
// columns of their own, [token][row], which the epilogue adds.  For a bf16 y these are the columns of
// the next tile's accumulator, which then starts after the epilogue; for a float32 y, of 128 tokens,
// there are columns for the three accumulators (see gdn_adapt.cu) and these, to which the accumulators of
// long sums are added too.  (That is slow beside the
// tensor core, whose operands take all of the shared memory's bandwidth: 15 us for a tile of 256 tokens
// with two adapters, whose k-blocks take 4.)
//
// Bound by the tensor pipe, 79 % active: 16384 tokens, 2048 -> 12352, in 488 us without adapters (1.70
// PFLOP/s), 555 in prompts of 1100 with adapters of rank 64 (of which the low side some 50), 706 in runs of
// 50.  777 float32 tokens in runs of 50, 2048 -> 5120: 47.0 us, a tile and its epilogue one after the other.
#include "gdn_adapt.cuh"

namespace gdn {
namespace {

using namespace adapt;

constexpr int kTeams = 3;      // of four warps (with four, a thread has 96 registers, which do not suffice)
constexpr int kWarps = 4 * kTeams;
constexpr int kHelpers = 32 * kWarps;
constexpr int kThreads = 64 + kHelpers + 32;
constexpr int kInfo = 8;  // tiles looked ahead

template <typename TO>
struct Cfg {
  static constexpr bool kF32 = sizeof(TO) == 4;
  static constexpr int kParts = kF32 ? 3 : 2;
  static constexpr int BT = kF32 ? 128 : 256;
  static constexpr int kAcc = kF32 ? 3 : 1;
  static constexpr int kRound = kAcc * kChain;  // k-blocks after which a float32 y's are taken out
  static constexpr int kStage = kTileW + BT / 2 * kBK * 2;
  static constexpr int kStages = 6;
  static constexpr int kScratch = kWarps * 16 * 33 * 4;
  static constexpr int kSmem = kStages * kStage + kScratch + 1024;
};

constexpr int kMany = -2, kGaveUp = -3, kMixed = -4;
// The adapters of a tile that are k-blocks of it.
__device__ __forceinline__ int adapters_of(int one) {
  return one >= 0 ? 1 : one <= kMixed ? kMixed - one : 0;
}

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t leader_addr(const void *p) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
  return a;
}
// to this CTA's shared memory, reported to a barrier of CTA 0
__device__ __forceinline__ void tma_load2_pair(void *dst, const CUtensorMap *m, int x, int y,
                                               uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(leader_bar)
      : "memory");
}
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// As if a copy of `bytes` had reported to the barrier.
__device__ __forceinline__ void complete_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void st_peer64(const void *p, int rank, int64_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.b64 [a], %2;\n\t}" ::"r"(smem_addr(p)),
      "r"(rank), "l"(v)
      : "memory");
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr),
               "r"(__float_as_uint(v))
               : "memory");
}

// Ranks e .. e + W / 2 - 1 of a row of B, zeros from `rank` on (what lies behind a row is not read).
// WHOLE: the rank is a multiple of W / 2.
template <int W, bool WHOLE>
__device__ __forceinline__ void load_b(const bf16 *row, int e, int rank, uint32_t *out) {
  if constexpr (WHOLE) {
    load_words<W>(row + (e < rank ? e : 0), out);
    if (e >= rank)
#pragma unroll
      for (int w = 0; w < W / 4; ++w) out[w] = 0;
  } else {
#pragma unroll
    for (int w = 0; w < W / 4; ++w) out[w] = 0;
#pragma unroll
    for (int j = 0; j < W / 2; ++j)
      if (e + j < rank)
        out[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[e + j] << (16 * (j & 1));
  }
}

// Run by the helpers (`warp` of them; `quad`: the TMEM lanes it may write, 32 quad ..): every third
// task.  Lane (r, c) of a fragment has rows r and r + 8 of B and token r of the task, for each W bytes
// the same ranks (W / 2 neighbours: the order of K does not matter); NL such loads at a time, HALVES
// times.  B stays in registers while the group does, and what the team's next task needs is on its way
// under a task's results, unless there are two halves.
template <int BT, int W, int NL, int HALVES, bool WHOLE, int PARTS>
__device__ __forceinline__ void expand(const AdaptArgs &g, const Groups<BT> &s, int warp, int quad,
                                       int n0, int tok0, float *scratch, uint32_t delta) {
  constexpr int kWords = W / 4;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, team = warp >> 2;
  const int ld = g.rank_pad();
  const int64_t part = (int64_t)g.tokens * ld;
  const bf16 *h0 = static_cast<const bf16 *>(g.h) + (int64_t)tok0 * ld + c * (W / 2);
  uint32_t b[2][NL][2][kWords], h[NL][PARTS][kWords];
  auto load_h = [&](int t, int half) {
    const bf16 *p = h0 + s.token[t][r] * ld + half * (NL * 2 * W);
#pragma unroll
    for (int l = 0; l < NL; ++l)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) load_words<W>(p + q * part + l * 2 * W, h[l][q]);
  };
  auto load_rows = [&](int group, int half) {
    const bf16 *b0 = static_cast<const bf16 *>(g.b) + (int64_t)s.adapter[group] * g.n_out * g.ld_b;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const bf16 *row = b0 + min(n0 + 32 * quad + 16 * m + 8 * y + r, g.n_out - 1) * g.ld_b;
#pragma unroll
        for (int l = 0; l < NL; ++l)
          load_b<W, WHOLE>(row, (half * NL + l) * 2 * W + c * (W / 2), g.rank, b[m][l][y]);
      }
  };
  int group = -1;
  auto load = [&](int t) {
    if (s.group[t] != group) load_rows(group = s.group[t], 0);
    load_h(t, 0);
  };
  if (HALVES == 1 && team < s.tasks) load(team);
  for (int t = team; t < s.tasks; t += kTeams) {
    float acc[2][PARTS][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[m][q][x] = 0.f;
#pragma unroll 1
    for (int half = 0; half < HALVES; ++half) {
      if (HALVES > 1) {
        load_rows(s.group[t], half);
        load_h(t, half);
      }
#pragma unroll
      for (int l = 0; l < NL; ++l)
#pragma unroll
        for (int w = 0; w < kWords; w += 2)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t a[4] = {b[m][l][0][w], b[m][l][1][w], b[m][l][0][w + 1],
                                   b[m][l][1][w + 1]};
#pragma unroll
            for (int q = 0; q < PARTS; ++q) mma16816(acc[m][q], a, h[l][q][w], h[l][q][w + 1]);
          }
    }
    if (HALVES == 1 && t + kTeams < s.tasks) load(t + kTeams);
    // from fragments to a row a lane
    __syncwarp();
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = acc[m][0][x] + acc[m][1][x];
        if constexpr (PARTS == 3) v += acc[m][2][x];
        scratch[(2 * c + (x & 1)) * 33 + 16 * m + 8 * (x >> 1) + r] = v;
      }
    __syncwarp();
    const int cols = s.tokens[t];
    for (int j = 0; j < cols; ++j) tmem_st1(delta + s.token[t][j], scratch[j * 33 + lane]);
  }
}

template <int BT, bool WHOLE, int PARTS>
__device__ __forceinline__ void expand_rank(const AdaptArgs &g, const Groups<BT> &s, int warp, int quad,
                                            int n0, int tok0, float *scratch, uint32_t delta) {
  if (g.rank <= 16)
    expand<BT, 8, 1, 1, WHOLE, PARTS>(g, s, warp, quad, n0, tok0, scratch, delta);
  else if (g.rank <= 32)
    expand<BT, 16, 1, 1, WHOLE, PARTS>(g, s, warp, quad, n0, tok0, scratch, delta);
  else if (g.rank <= 64)
    expand<BT, 16, 2, 1, WHOLE, PARTS>(g, s, warp, quad, n0, tok0, scratch, delta);
  else
    expand<BT, 16, 2, 2, WHOLE, PARTS>(g, s, warp, quad, n0, tok0, scratch, delta);
}

// Outputs row0 .. row0 + 31 of tokens tok .. tok + live - 1 (at most 16) by themselves, a warp: W x with
// mma.sync (see gdn_adapt_low.cu for the loads), and what each token's own adapter adds.  The tile's
// adapters are list[0 .. count).  Into out [token][33].
template <int PARTS>
__device__ __forceinline__ void again(const AdaptArgs &g, const int *list, int count, int row0, int tok,
                                   int live, float *out) {
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const bf16 *x[2], *w[2][2];  // (rows that are not there: any, their results are dropped)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i] = static_cast<const bf16 *>(g.x) + (tok + min(8 * i + r, live - 1)) * g.ld_x;
#pragma unroll
    for (int y = 0; y < 2; ++y)
      w[i][y] = static_cast<const bf16 *>(g.w) + min(row0 + 16 * i + 8 * y + r, g.n_out - 1) * g.ld_w;
  }
  float sum[2][2][4] = {};
  for (int k0 = 0; k0 < g.hidden; k0 += 256) {  // (short chains: these sums are cut off too)
    float acc[2][2][4] = {};
    const int end = min(k0 + 256, g.hidden);
#pragma unroll 2
    for (int k = k0; k < end; k += 32) {
      uint4 a[2][2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[i] = load8<false>(x[i], k + 8 * c, g.hidden);
#pragma unroll
        for (int y = 0; y < 2; ++y) a[i][y] = load8<false>(w[i][y], k + 8 * c, g.hidden);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t f0[4] = {a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y};
        const uint32_t f1[4] = {a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mma16816(acc[m][i], f0, b[i].x, b[i].y);
          mma16816(acc[m][i], f1, b[i].z, b[i].w);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[m][i][e] += acc[m][i][e];
  }
  kv::dependent_wait();  // h
  // what the adapters add: all of one to every token, and kept where it is the token's own
  const int ld = g.rank_pad(), id = lane < live ? token_id(g, tok + lane) : -1;
  const int64_t part = (int64_t)g.tokens * ld;
  for (int j = 0; j < count; ++j) {
    const uint32_t own = __ballot_sync(0xffffffffu, id >= 0 && id == list[j]);
    if (own == 0) continue;
    float acc[2][2][4] = {};
    for (int k = 8 * c; k - 8 * c < g.rank; k += 32) {
      uint4 a[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int n = min(row0 + 16 * i + 8 * y + r, g.n_out - 1);
          a[i][y] = load8<false>(
              static_cast<const bf16 *>(g.b) + ((int64_t)list[j] * g.n_out + n) * g.ld_b, k, g.rank);
        }
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bf16 *h = static_cast<const bf16 *>(g.h) + (j * PARTS + p) * part +
                          (int64_t)(tok + min(8 * i + r, live - 1)) * ld;
          const uint4 b = load8<true>(h, k, ld);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t f0[4] = {a[m][0].x, a[m][1].x, a[m][0].y, a[m][1].y};
            const uint32_t f1[4] = {a[m][0].z, a[m][1].z, a[m][0].w, a[m][1].w};
            mma16816(acc[m][i], f0, b.x, b.y);
            mma16816(acc[m][i], f1, b.z, b.w);
          }
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (own >> (8 * i + 2 * c + (e & 1)) & 1) sum[m][i][e] += acc[m][i][e];
  }
  __syncwarp();
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[(8 * i + 2 * c + (e & 1)) * 33 + 16 * m + 8 * (e >> 1) + r] = sum[m][i][e];
  __syncwarp();
}

// 16 tokens' outputs n, a lane per output: two neighbouring lanes exchange, so that each stores two
// outputs of every other token.
__device__ __forceinline__ void store_rows(bf16 *y, int64_t ld, int n, int n_out, int live,
                                           const float *v) {
  const int odd = n & 1;
  bf16 *p = y + odd * ld + (n - odd);
#pragma unroll
  for (int j = 0; j < 16; j += 2, p += 2 * ld) {
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(other, v[j + 1])
                                 : __floats2bfloat162_rn(v[j], other);
    if (j + odd >= live) continue;
    if (n - odd + 1 < n_out)
      *reinterpret_cast<__nv_bfloat162 *>(p) = w;
    else if (n - odd < n_out)
      *p = w.x;
  }
}

// 16 tokens' results of this lane's row, from column c of the accumulators on; `delta`: what is to be
// added, if `summed`.  kbs: the tile's k-blocks.
template <typename TO>
__device__ __forceinline__ void load_results(uint32_t acc, uint32_t delta, bool summed, int kbs, int c,
                                             float *v) {
  using C = Cfg<TO>;
  constexpr int BT = C::BT;
  if constexpr (C::kF32) {
    float u[32];
    tc::tmem_ld32(acc + c, acc + BT + c, v);
    const int last = (kbs - 1) % C::kRound + 1;
    if (last > 1)  // (an accumulator that no k-block of the round has come to holds anything)
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += v[16 + j];
    if (summed)
      tc::tmem_ld32(acc + 2 * BT + c, delta + c, u);
    else
      tc::tmem_ld16(acc + 2 * BT + c, u);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (last > 2) v[j] += u[j];
      if (summed) v[j] += u[16 + j];
    }
  } else if (summed) {
    tc::tmem_ld32(acc + c, delta + c, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += v[16 + j];
  } else {
    tc::tmem_ld16(acc + c, v);
  }
}

// Outputs n of tokens tok .. tok + min(live, 16) - 1.
__device__ __forceinline__ void store_results(const AdaptArgs &g, float *y, int tok, int live, int n,
                                              const float *v) {
  if (n >= g.n_out) return;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < live) y[(int64_t)(tok + j) * g.ld_y + n] = v[j];
}
__device__ __forceinline__ void store_results(const AdaptArgs &g, bf16 *y, int tok, int live, int n,
                                              const float *v) {
  store_rows(y + (int64_t)tok * g.ld_y, g.ld_y, n, g.n_out, live, v);
}

__device__ __forceinline__ float result(float v) { return v; }
__device__ __forceinline__ float result(bf16 v) { return __bfloat162float(v); }

// After a warp's last tile, if there were results that are not finite in mixed tiles: they are computed
// again, of the `stored` tiles.  (Within the loop over the tiles the call would cost it registers, and the
// products would wait.)
template <typename TO>
__device__ __noinline__ void results_again(const AdaptArgs &g, int stored, int *list, float *own) {
  using C = Cfg<TO>;
  const int lane = threadIdx.x & 31, quad = threadIdx.x >> 5 & 3, side = ((int)(threadIdx.x >> 5) - 2) >> 2;
  const int n_tiles = (g.n_out + 2 * kBM - 1) / (2 * kBM);
  TO *y = static_cast<TO *>(g.y);
  int64_t t = blockIdx.x >> 1;
  for (int i = 0; i < stored; ++i, t += gridDim.x >> 1) {
    const int tok0 = (int)(t / n_tiles) * C::BT, live = min(C::BT, g.tokens - tok0);
    const int row0 = (int)(t % n_tiles) * 2 * kBM + (int)cluster_rank() * kBM + 32 * quad;
    __syncwarp();
    const int count = tile_groups(g, tok0, live, list);
    __syncwarp();
    if (row0 >= g.n_out || count == 0 || count > kPlanes) continue;
    bool whole = true;  // no token without an adapter
    for (int j = lane; j < live; j += 32) whole = whole && token_id(g, tok0 + j) >= 0;
    if (count == 1 && __all_sync(0xffffffffu, whole)) continue;
    for (int c = 16 * side; c < live; c += 16 * kTeams) {
      TO *at = y + (int64_t)(tok0 + c) * g.ld_y + min(row0 + lane, g.n_out - 1);
      const int steps = min(16, live - c);
      bool finite = true;
      for (int j = 0; j < steps; ++j) finite = finite && fabsf(result(at[j * g.ld_y])) < INFINITY;
      if (__all_sync(0xffffffffu, finite)) continue;
      again<C::kParts>(g, list, count, row0, tok0 + c, steps, own);
      if (row0 + lane < g.n_out)
        for (int j = 0; j < steps; ++j)
          if (!(fabsf(result(at[j * g.ld_y])) < INFINITY))
            Elem<TO>::store1(at + j * g.ld_y, own[j * 33 + lane]);
      __syncwarp();
    }
  }
}

// Among the helpers: whether all say so.
__device__ __forceinline__ bool helpers_and(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kHelpers)
      : "memory");
  return r != 0;
}

template <typename TO>
__global__ void __launch_bounds__(kThreads, 1)
    adapt_pair_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                      const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mh,
                      const __grid_constant__ AdaptArgs g) {
  using C = Cfg<TO>;
  constexpr int S = C::kStages, BT = C::BT;
  extern __shared__ unsigned char dsm_raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2], info_full[kInfo],
      info_empty[kInfo], round_full, round_taken, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ uint32_t s_limit;  // of the waits
  __shared__ int s_info[kInfo], s_list[kInfo][kPlanes], s_again[kWarps][kPlanes];
  __shared__ float s_gone;      // one of the two gave up
  __shared__ int64_t s_issued, s_other;  // k-blocks whose copies were started, here and (CTA 0) by the other
  __shared__ Groups<BT> s_groups;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~uintptr_t(1023));
  auto tile_w = [&](int s) { return smem + s * C::kStage; };
  auto tile_x = [&](int s) { return smem + s * C::kStage + kTileW; };
  float *scratch = reinterpret_cast<float *>(smem + S * C::kStage);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int n_tiles = (g.n_out + 2 * kBM - 1) / (2 * kBM), t_tiles = (g.tokens + BT - 1) / BT;
  const int64_t tiles = (int64_t)n_tiles * t_tiles;
  const int plain = (g.hidden + kBK - 1) / kBK, chunks = (g.rank + kBK - 1) / kBK;
  // (test hooks: in every other pair a barrier waits for what no one sends, CTA 0's first copies', or that
  // of the first tile's adapters in CTA 0 or 1)
  const uint32_t hook = pair & 1 ? g.test_flags : 0;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kWarps);
    }
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&info_full[i], i == 0 && hook & GDN_TEST_ADAPT_SIDE_TIMEOUT && (pair >> 1 & 1) == rank ? 2 : 1);
      mbar_init(&info_empty[i], kWarps);
    }
    mbar_init(&round_full, 1);
    mbar_init(&round_taken, 2 * kWarps);
    mbar_init(&drain, 1);
    s_limit = patience(g);
    s_gone = 0.f;
    mbar_fence_init();
    if (hook & GDN_TEST_ADAPT_WAIT_TIMEOUT) mbar_expect_tx(&full[0], 16);
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile uint32_t *limit = &s_limit;
  auto fail = [&]() {
    *limit = 0;
    raise_error(g.err, GDN_DEVERR_TIMEOUT);
  };
  // the adapter that all tokens of the pair's i-th tile have, or -1: none has any, kMany: more than there
  // are planes for, kGaveUp: a wait did, kMixed - n: n (s_list)
  auto tile_info = [&](int i) {
    if (!wait(&info_full[i % kInfo], (i / kInfo) & 1, limit)) return kGaveUp;
    return *reinterpret_cast<volatile int *>(&s_info[i % kInfo]);
  };

  if (warp == 0 && lane == 0) {
    // producer
    int s = 0;
    uint32_t round = 0;
    int64_t u = 0;
    bool good = true, waited = false;
    int i = 0;
    for (int64_t t = pair; t < tiles && good; t += pairs, ++i) {
      const int tok0 = (int)(t / n_tiles) * BT + rank * (BT / 2);
      const int n0 = (int)(t % n_tiles) * 2 * kBM + rank * kBM;
      const int one = tile_info(i);
      if (one == kGaveUp) {
        good = false;
        break;
      }
      const int kbs = plain + adapters_of(one) * chunks * C::kParts;
      for (int kb = 0; kb < kbs; ++kb, ++u, s = s + 1 == S ? 0 : s + 1) {
        if (s == 0 && u > S) round ^= 1;  // (the first round waits for nothing, the second for phase 0)
        if (u >= S && !wait(&empty[s], round, limit)) {
          good = false;
          break;
        }
        const uint32_t bar = leader_addr(&full[s]);
        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
        if (kb < plain) {
          tma_load2_pair(tile_w(s), &mw, kb * kBK, n0, bar);
          tma_load2_pair(tile_x(s), &mx, kb * kBK, tok0, bar);
        } else {
          // (rows of h behind the last token are another part's: columns that are not stored)
          const int e = kb - plain, p = e % C::kParts, c = e / C::kParts % chunks,
                    j = e / C::kParts / chunks;
          const int id = one >= 0 ? one : s_list[i % kInfo][j];
          tma_load2_pair(tile_w(s), &mb, c * kBK, id * g.n_out + n0, bar);
          if (!waited) {
            kv::dependent_wait();
            asm volatile("fence.proxy.async.global;" ::: "memory");  // plain stores, read by TMA
            waited = true;
          }
          tma_load2_pair(tile_x(s), &mh, c * kBK, (j * C::kParts + p) * g.tokens + tok0, bar);
        }
      }
    }
    s_issued = u;
    if (!good) fail();
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // MMA issuer
    constexpr uint32_t idesc = tc::idesc_bf16(2 * kBM, BT);
    int s = 0;
    uint32_t round = 0;
    bool good = true;
    int i = 0, before = -1;  // the tile before: it has no adapters
    uint32_t rounds = 0;     // of the accumulators, that were taken out
    for (int64_t t = pair; t < tiles && good; t += pairs, ++i) {
      const int one = tile_info(i);
      // The accumulators' columns are free once the epilogue of tile i - 2 is done, or of tile i - 1
      // where they are the same or held its adapters' part.
      auto free_after = [&](int last) {
        return last < 0 || wait(&acc_empty[last & 1], (uint32_t)((last >> 1) & 1), limit);
      };
      if (one == kGaveUp || !free_after(C::kF32 || before == kMany ? i - 1 : i - 2)) {
        good = false;
        break;
      }
      before = one;
      tc::fence_after_sync();
      const uint32_t base = C::kF32 ? tmem : tmem + (uint32_t)(i & 1) * BT;
      int turn = 0, in = 0;  // of the accumulators; k-blocks of the round
      // the next k-block's products; a loop round it has 256 cycles
      auto block = [&](int steps) {
        if (C::kF32 && in == C::kRound) {
          commit_pair(&round_full);
          if (!wait(&round_taken, rounds++ & 1, limit)) return false;
          tc::fence_after_sync();
          turn = in = 0;
        }
        const uint32_t acc = base + (uint32_t)turn * BT;
        const bool fresh = in++ < C::kAcc;
        turn = turn + 1 == C::kAcc ? 0 : turn + 1;
        if (!wait(&full[s], round, limit)) return false;
        tc::fence_after_sync();
        const uint32_t a = smem_addr(tile_w(s)), b = smem_addr(tile_x(s));
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          if (kk < steps)
            mma_pair(acc, tc::smem_desc_sw128(a + 32 * kk), tc::smem_desc_sw128(b + 32 * kk), idesc,
                     !fresh || kk > 0 ? 1u : 0u);
        commit_pair(&empty[s]);
        if (++s == S) s = 0, round ^= 1;
        return true;
      };
      for (int kb = 0; kb < plain && good; ++kb) good = block(kBK / 16);
      for (int j = adapters_of(one); j > 0; --j)
        for (int c = 0; c < chunks; ++c)
          for (int p = 0; p < C::kParts && good; ++p)
            good = block(min(kBK, g.rank16() - c * kBK) / 16);
      if (good) commit_pair(&acc_full[i & 1]);
    }
    if (!good) fail();
  } else if (warp == 2 + kWarps) {
    // scout
    int i = 0;
    bool good = true;
    for (int64_t t = pair; t < tiles && good; t += pairs, ++i) {
      const int tok0 = (int)(t / n_tiles) * BT, live = min(BT, g.tokens - tok0);
      if (i >= kInfo)
        good = __all_sync(0xffffffffu,
                          wait(&info_empty[i % kInfo], ((i / kInfo) - 1) & 1, limit));
      if (!good) break;
      const int n = tile_groups(g, tok0, live, s_list[i % kInfo]);
      bool whole = true;  // no token without an adapter
#pragma unroll
      for (int j = 0; j < BT / 32; ++j)
        if (32 * j + lane < live) whole = whole && token_id(g, tok0 + 32 * j + lane) >= 0;
      whole = __all_sync(0xffffffffu, whole);
      if (lane == 0) {
        *reinterpret_cast<volatile int *>(&s_info[i % kInfo]) =
            n == 0 ? -1 : n == 1 && whole ? s_list[i % kInfo][0] : n > kPlanes ? kMany : kMixed - n;
        mbar_arrive(&info_full[i % kInfo]);
      }
    }
    if (!good) fail();
  } else if (warp >= 2 && warp < 2 + kWarps) {
    const int quad = warp & 3, side = (warp - 2) >> 2;
    const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16);
    TO *y = static_cast<TO *>(g.y);
    int i = 0;
    uint32_t rounds = 0;
    bool good = true, odd = false;  // odd: mixed tiles had results that are not finite
    int stored = 0;
    for (int64_t t = pair; t < tiles; t += pairs, ++i) {
      const int tok0 = (int)(t / n_tiles) * BT, live = min(BT, g.tokens - tok0);
      const int n0 = (int)(t % n_tiles) * 2 * kBM + rank * kBM, n = n0 + 32 * quad + lane;
      // (the helpers meet in barriers: they give up together, or not yet)
      const int one = good ? tile_info(i) : kGaveUp;
      if (!helpers_and(one != kGaveUp)) {
        fail();
        break;
      }
      tc::fence_after_sync();  // all have read the tile before
      const uint32_t acc = mine + (C::kF32 ? 0u : (uint32_t)(i & 1) * BT);
      const uint32_t delta = mine + (C::kF32 ? 3u * BT : (uint32_t)((i & 1) ^ 1) * BT);
      if (one == kMany) {
        const float zero[16] = {};  // what tokens without an adapter get
#pragma unroll 1
        for (int c = 16 * side; c < BT; c += 16 * kTeams) tc::tmem_st16(delta + c, zero);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        if (tid - 64 < BT) s_groups.id[tid - 64] = token_id(g, tok0 + tid - 64);
        helpers_sync<kHelpers>();
        find_groups<BT, kHelpers>(s_groups);
        tc::fence_after_sync();
        kv::dependent_wait();  // h
        float *sc = scratch + (warp - 2) * 16 * 33;
        if (n0 < g.n_out) {
          if (g.rank % 8 == 0)
            expand_rank<BT, true, C::kParts>(g, s_groups, warp - 2, quad, n0, tok0, sc, delta);
          else
            expand_rank<BT, false, C::kParts>(g, s_groups, warp - 2, quad, n0, tok0, sc, delta);
        }
        tc::tmem_st_wait();
        tc::fence_before_sync();
        helpers_sync<kHelpers>();
      }
      // the accumulators of a long sum, taken out into the columns of `delta`
      const int kbs = plain + adapters_of(one) * chunks * C::kParts;
      if constexpr (C::kF32)
        for (int k = C::kRound; k < kbs && good; k += C::kRound, ++rounds) {
          good = __all_sync(0xffffffffu, wait(&round_full, rounds & 1, limit));
          if (!good) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int c = 16 * side; c < live; c += 16 * kTeams) {
            float v[32], u[32];
            tc::tmem_ld32(acc + c, acc + BT + c, v);
            if (one == kMany || k > C::kRound) {
              tc::tmem_ld32(acc + 2 * BT + c, delta + c, u);
#pragma unroll
              for (int j = 0; j < 16; ++j) u[j] += u[16 + j];
            } else {
              tc::tmem_ld16(acc + 2 * BT + c, u);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += v[16 + j] + u[j];
            tc::tmem_st16(delta + c, v);
          }
          tc::tmem_st_wait();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) arrive_leader(&round_taken);
        }
      good = good &&
             __all_sync(0xffffffffu, wait(&acc_full[i & 1], (i >> 1) & 1, limit));
      if (!good) {
        fail();
        continue;
      }
      tc::fence_after_sync();
      const bool summed = one == kMany || (C::kF32 && kbs > C::kRound);
#pragma unroll 1
      for (int c = 16 * side; c < live; c += 16 * kTeams) {
        float v[32];
        load_results<TO>(acc, delta, summed, kbs, c, v);
        if (one <= kMixed) {
          bool finite = true;
          if (live - c >= 16) {
#pragma unroll
            for (int j = 0; j < 16; ++j) finite = finite && fabsf(v[j]) < INFINITY;
          } else {  // (columns behind the last token hold anything)
#pragma unroll
            for (int j = 0; j < 16; ++j) finite = finite && (c + j >= live || fabsf(v[j]) < INFINITY);
          }
          odd = odd || (!finite && n < g.n_out);
        }
        store_results(g, y, tok0 + c, live - c, n, v);
      }
      ++stored;
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&info_empty[i % kInfo]);
        arrive_leader(&acc_empty[i & 1]);
      }
    }
    if (__any_sync(0xffffffffu, odd))
      results_again<TO>(g, stored, s_again[warp - 2], scratch + (warp - 2) * 16 * 33);
  }
  // (the leader's products read the other CTA's shared memory, and its commits arrive there)
  tc::fence_before_sync();
  __syncthreads();
  if (tid == 0 && *limit == 0)
    for (int p = 0; p < 2; ++p) st_peer(&s_gone, p, 1.f);
  cluster_sync();
  if (s_gone != 0.f) {  // copies and products still in flight end before the pair does
    if (rank == 1 && tid == 0) st_peer64(&s_other, 0, s_issued);
    cluster_sync();
    if (tid == 32) {
      if (rank == 0) commit_pair(&drain);
      mbar_wait_bounded(&drain, 0, patience(g));
    }
    if (rank == 0 && tid == 0) {
      // The two may have stopped at different k-blocks.  Of what both started, CTA 0's barriers await both;
      // of what only one did, its half: CTA 0 awaits the other's too, or nothing yet.
      const int64_t both = min(s_issued, s_other), any = max(s_issued, s_other);
      for (int64_t q = max((int64_t)0, both - S); q < any; ++q) {
        uint64_t *bar = &full[q % S];
        if (q >= both && s_issued > both) complete_tx(bar, C::kStage);
        if (q >= both && s_issued == both) mbar_arrive_expect_tx(bar, C::kStage);
        mbar_wait_bounded(bar, (uint32_t)((q / S) & 1), patience(g));
      }
    }
    cluster_sync();
  }
  if (warp == 1) {
    tc::fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  }
  // what follows on the stream waits for this kernel only: the low side is complete too
  kv::dependent_wait();
}

template <typename TO>
cudaError_t launch(const AdaptArgs &g, cudaStream_t s) {
  using C = Cfg<TO>;
  CUtensorMap mw, mx, mb, mh;
  const int64_t ld = g.rank_pad();
  if (!encode_rows(&mw, g.w, g.n_out, g.hidden, g.ld_w, kBM) ||
      !encode_rows(&mx, g.x, g.tokens, g.hidden, g.ld_x, C::BT / 2) ||
      !encode_rows(&mb, g.b, (int64_t)g.n_adapters * g.n_out, g.rank, g.ld_b, kBM) ||
      !encode_rows(&mh, g.h, (int64_t)kPlanes * C::kParts * g.tokens, ld, ld, C::BT / 2))
    return cudaErrorNotSupported;
  static std::atomic<uint64_t> seen{0};
  const cudaError_t e = kv::allow_smem(adapt_pair_kernel<TO>, C::kSmem, g.device, seen);
  if (e != cudaSuccess) return e;
  const int64_t tiles =
      (int64_t)((g.n_out + 2 * kBM - 1) / (2 * kBM)) * ((g.tokens + C::BT - 1) / C::BT);
  const int pairs = (int)(tiles < g.sm_count / 2 ? tiles : g.sm_count / 2);
  return kv::launch(adapt_pair_kernel<TO>, dim3((unsigned)(2 * pairs)), kThreads, C::kSmem, s, 2, mw,
                    mx, mb, mh, g);
}

}  // namespace

cudaError_t launch_adapt_pair(const AdaptArgs &g, cudaStream_t s) {
  return g.y_dtype == GDN_F32 ? launch<float>(g, s) : launch<bf16>(g, s);
}

}  // namespace gdn
