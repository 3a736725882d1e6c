// The low side of the adapters: h[t] = scale[a] A[a] x[t], a = ids[t], summed in float32 and stored as
// bf16 parts that add up to it.
//
// Bound by the bytes of the A in use (a decode step) or of x (prompts), so the products go where the
// data can be used without a detour: mma.sync takes both operands from registers, and those are
// loaded straight from global memory, 16 bytes a lane.  The order of k within a product does not
// matter, so a lane's 16 bytes -- 8 neighbours in k -- are fed to two products as they come.
// (These products are 3 % of a prompt's; the tensor cores that read shared memory are for the
// projection itself.)  16384 tokens, rank 64, take 54 us, for 268 MB through L2.
//
// A CTA takes a window of 16 * MT tokens, the adapters of which it finds by comparing the ids, and
// 8 * NT ranks; its 8 warps split the sum over k, joined in shared memory in a fixed order.  Where
// a window may have many adapters and there are few windows, several CTAs share it (blockIdx.y), each
// taking every gridDim.y-th adapter.
#include "gdn_adapt.h"
#include "gdn_common.cuh"
#include "gdn_kv.cuh"
#include "gdn_mma.cuh"

#include "gdn_adapt_tile.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;

// AHEAD: steps of 64 k whose loads a warp has in flight.  (With the ends of odd rows looked at in
// every load the code was so long that fetching it took longer than the work.)
template <int MT, int NT, int AHEAD, bool WHOLE, bool PLANES>
__global__ void __launch_bounds__(32 * kWarps, MT * NT == 8 ? 2 : 1) low_kernel(AdaptArgs g) {
  constexpr int kTok = 16 * MT, kRanks = 8 * NT;
  extern __shared__ float s_part[];  // [kWarps][kTok][kRanks]
  __shared__ int s_id[kTok], s_lead[kTok], s_n;
  __shared__ int s_plane[PLANES ? kTok : 1];
  __shared__ int s_tile[kPlanes], s_tile_n;  // PLANES: the adapters of the window's tile
  kv::dependent_wait();
  // the projection may start loading what no kernel before this one writes
  kv::dependents_may_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tok0 = blockIdx.x * kTok, rank0 = blockIdx.z * kRanks;
  const int row = lane >> 2, col = lane & 3;
  // (a row behind the last token: any row, its result is dropped)
  const bf16 *xrow[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
      xrow[m][hh] = static_cast<const bf16 *>(g.x) +
                    min(tok0 + 16 * m + 8 * hh + row, g.tokens - 1) * g.ld_x;
  uint4 xv[AHEAD][MT][2][2];
  auto load_x = [&](int k0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            xv[i][m][hh][c] = load8<WHOLE>(xrow[m][hh], k0 + 64 * kWarps * i + 32 * c + 8 * col, g.hidden);
  };
  // x is on its way before the ids are known
  load_x(64 * warp);
  int own = -1;
  if (tid < kTok) {
    if (tok0 + tid < g.tokens) own = g.ids[tok0 + tid];
    if (own < -1 || own >= g.n_adapters) {
      if (blockIdx.y + blockIdx.z == 0) raise_error(g.err, GDN_DEVERR_ADAPTER);
      own = -1;
    }
    s_id[tid] = own;
  }
  __syncthreads();
  if (warp == 0) {  // the window's adapters, in the order of their first tokens
    int n = 0;
    for (int base = 0; base < kTok; base += 32) {
      const int i = base + lane;
      const int id = i < kTok ? s_id[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      bool lead = id >= 0 && __ffs(same) - 1 == lane;
      for (int j = 0; j < base; ++j) lead = lead && s_id[j] != id;
      const uint32_t m = __ballot_sync(0xffffffffu, lead);
      if (lead) s_lead[n + __popc(m & ((1u << lane) - 1))] = id;
      n += __popc(m);
    }
    if (lane == 0) s_n = n;
  }
  if (PLANES && warp == 1) {
    const int t0 = tok0 / g.tile * g.tile;
    const int n = tile_groups(g, t0, min(g.tile, g.tokens - t0), s_tile);
    if (lane == 0) s_tile_n = n;
  }
  __syncthreads();
  const int64_t part_words = (int64_t)g.tokens * (g.rank_pad() / 2);
  if (PLANES) {
    if (tid < kTok) {
      int plane = 0;
      if (s_id[tid] < 0)
        plane = -1;
      else if (s_tile_n <= kPlanes)
        while (s_tile[plane] != s_id[tid]) ++plane;
      s_plane[tid] = plane;
    }
    __syncthreads();
    // zeros in the planes of the tile's other adapters, shared by the CTAs of a window
    if (s_tile_n <= kPlanes) {
      constexpr int kVecs = kRanks / 8;
      const int rows = kTok * g.parts() * kVecs;
      for (int j = blockIdx.y; j < s_tile_n; j += gridDim.y)
        for (int i = tid; i < rows; i += 32 * kWarps) {
          const int v = i % kVecs, t = i / kVecs % kTok, p = i / (kVecs * kTok), r = rank0 + 8 * v;
          if (s_plane[t] == j || tok0 + t >= g.tokens || r >= g.rank_pad()) continue;
          reinterpret_cast<uint4 *>(static_cast<uint32_t *>(g.h) +
                                    (j * g.parts() + p) * part_words)[
              ((int64_t)(tok0 + t) * g.rank_pad() + r) / 8] = make_uint4(0, 0, 0, 0);
        }
    }
  }
  const int rank_pad = g.rank_pad(), parts = g.parts();
  for (int gi = blockIdx.y; gi < s_n; gi += gridDim.y) {
    const int id = s_lead[gi];
    const float scale = g.scale[id];
    const bf16 *a = static_cast<const bf16 *>(g.a) + (int64_t)id * g.rank * g.ld_a;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][n][e] = 0.f;
    for (int k0 = 64 * warp; k0 < g.hidden; k0 += 64 * kWarps * AHEAD) {
      uint4 av[AHEAD][NT][2];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = rank0 + 8 * n + row, k = k0 + 64 * kWarps * i + 32 * c + 8 * col;
            av[i][n][c] = r < g.rank ? load8<WHOLE>(a + r * g.ld_a, k, g.hidden) : make_uint4(0, 0, 0, 0);
          }
      // (the first x of the first adapter are here already)
      if (gi != blockIdx.y || k0 != 64 * warp) load_x(k0);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const uint4 u = xv[i][m][0][c], v = xv[i][m][1][c];
            const uint32_t f0[4] = {u.x, v.x, u.y, v.y}, f1[4] = {u.z, v.z, u.w, v.w};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816(acc[m][n], f0, av[i][n][c].x, av[i][n][c].y);
              mma16816(acc[m][n], f1, av[i][n][c].z, av[i][n][c].w);
            }
          }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          *reinterpret_cast<float2 *>(
              &s_part[(warp * kTok + 16 * m + 8 * hh + row) * kRanks + 8 * n + 2 * col]) =
              make_float2(acc[m][n][2 * hh], acc[m][n][2 * hh + 1]);
    __syncthreads();
    for (int i = tid; i < kTok * kRanks / 2; i += 32 * kWarps) {  // two ranks a thread
      const int t = 2 * i / kRanks, r = rank0 + 2 * i % kRanks;
      if (s_id[t] != id || r >= rank_pad) continue;
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = *reinterpret_cast<const float2 *>(&s_part[w * kTok * kRanks + 2 * i]);
        sum.x += v.x, sum.y += v.y;
      }
      // (zeros beyond the rank, whatever the scale is)
      float x = r < g.rank ? sum.x * scale : 0.f, y = r + 1 < g.rank ? sum.y * scale : 0.f;
      uint32_t *h = static_cast<uint32_t *>(g.h) + ((int64_t)(tok0 + t) * rank_pad + r) / 2 +
                    (PLANES ? s_plane[t] * parts * part_words : 0);
      for (int p = 0; p < parts; ++p) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&v);
        h[p * part_words] = w;
        const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
        // (what is infinite or NaN is the first part alone)
        x = fabsf(lo) < INFINITY ? x - lo : 0.f;
        y = fabsf(hi) < INFINITY ? y - hi : 0.f;
      }
    }
    __syncthreads();
  }
}

template <int MT, int NT, int AHEAD, bool WHOLE, bool PLANES>
cudaError_t launch(const AdaptArgs &g, int others, cudaStream_t s) {
  constexpr int smem = kWarps * 16 * MT * 8 * NT * 4;
  static std::atomic<uint64_t> seen{0};
  const cudaError_t e = kv::allow_smem(low_kernel<MT, NT, AHEAD, WHOLE, PLANES>, smem, g.device, seen);
  if (e != cudaSuccess) return e;
  const int windows = (g.tokens + 16 * MT - 1) / (16 * MT);
  const int parts = (g.rank_pad() + 8 * NT - 1) / (8 * NT);
  // CTAs that share a window: as many as it may have adapters, but no more than two an SM in all (with
  // four, of which most find nothing to do, 1024 tokens in prompts took 56.6 us instead of 51.3)
  const int64_t room = (int64_t)2 * g.sm_count / ((int64_t)windows * parts);
  int share = (int)(room < 1 ? 1 : room > 16 * MT ? 16 * MT : room);
  // A CTA of the projection finds no room beside one of these.  So these take the SMs that it leaves, if
  // that is kLeast for a window at least (fewer, and a window's adapters take too long one after the
  // other), else one an SM: 64 tokens with an adapter each, 2048 -> 12352, 16 for a window 24.5 us, 13
  // 21.7; 128 with 64 adapters, 2048 -> 5120, 16 22.7, 8 19.7; 64 of rank 64, 16 40.8, 8 39.5, 4 42.0.
  constexpr int kLeast = 8;
  if (!PLANES && share > kLeast) {
    const int64_t spare = (g.sm_count - others) / ((int64_t)windows * parts);
    const int64_t all = g.sm_count / ((int64_t)windows * parts);
    const int64_t fit = spare >= kLeast ? spare : all >= kLeast ? all : kLeast;
    if (fit < share) share = (int)fit;
  }
  return kv::launch(low_kernel<MT, NT, AHEAD, WHOLE, PLANES>, dim3((unsigned)windows, (unsigned)share, (unsigned)parts),
                    32 * kWarps, smem, s, 1, g);
}

}  // namespace

// Few tokens: windows of 16, for parallel loads of A; many: windows of 32, that read A less often, two
// CTAs an SM, so that one's loads cover the other's sums (with the projection and four CTAs an SM in
// all, 1024 in prompts, 2048 -> 12352: windows of 16 59.0 us, of 32 56.2, of 64 61.8; 16384: 625, 563, 572).
constexpr int kFewWindows = 512;

cudaError_t launch_adapt_low(const AdaptArgs &g, int others, cudaStream_t s) {
  if (g.tile > 0)
    return g.hidden % 8 != 0         ? launch<1, 2, 1, false, true>(g, others, s)
           : g.tokens <= kFewWindows ? launch<1, 2, 4, true, true>(g, others, s)
                                     : launch<2, 4, 1, true, true>(g, others, s);
  return g.hidden % 8 == 0 ? launch<1, 2, 4, true, false>(g, others, s)
                           : launch<1, 2, 1, false, false>(g, others, s);
}

}  // namespace gdn
