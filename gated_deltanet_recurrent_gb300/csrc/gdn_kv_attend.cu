// Causal grouped-query attention over the 8-bit KV cache: single tokens,
// drafts, and every call in float32 (the long bf16 calls go to
// gdn_kv_prompt.cu).
//
// Mathematics.  With value codes c_j, V scale 2^e_j and scores x_j = scale *
// log2(e) * q.k_j, the output is
//     o = sum_j 2^(x_j + e_j - M) c_j / sum_j 2^(x_j - M)
// for any M.  M follows the running maximum of y_j = x_j + e_j, so the weights
// 2^(y_j - M) that multiply the codes are well scaled whatever the V scales
// are, and can be rounded to binary16; the codes are exact in binary16.  The
// denominator sums 2^(y_j - M) * 2^-e_j in float32 (pages whose e lies far from
// the others' are treated apart, see gdn_kv.cuh).  M is raised only when some
// y_j exceeds it by more than 7, which saves most of the reductions and
// rescalings; it is a whole number, so that y_j - M, from one fused multiply-add,
// is rounded at its own size and not at that of y_j.  The weights are lifted by
// 2^8: the largest is between 2^7 and 2^15, and those down to 2^-21 of it keep
// binary16's full precision.  Queries are scaled by a power of two per row to lie
// in [1, 2) at their largest (rows from 2^117 on: up to 2^12) and rounded to binary16
// (exact for bf16), or split into two binary16 parts (float32).
//
// Work.  HBM-bound: each KV head's codes are read once for all its query rows.
// A unit is 8 * NT query rows (tokens x the query heads of one KV head) of one
// sequence against its whole context, in tiles of 64 tokens, 16 per warp:
//   S^T (16 tokens x 8 rows) = K Q^T and O^T (d x 8 rows) += V^T P^T by
//   mma.sync m16n8k16, which wants the small side as N = 8: the query rows of
//   a decode step fill it, where a 128-row tcgen05 tile would be 1/16 full.
// Each warp has its own ring of 16-token stages that one lane fills with tensor
// copies (16 rows of 128 bytes, 128-byte swizzle), so what is in flight takes no
// registers and no warp waits for another.  Which token is which k index, and
// which d which row, is free as long as both operands agree: the A operands of
// both products are 16-byte (d = 64: 8-byte) shared-memory reads of rows as they
// lie, and V needs no transposition beyond one byte permutation that the
// conversion to binary16 does anyway.  Row r of the products is token perm(r),
// an order in which these reads meet no bank twice under the swizzle.
//
// Split.  All tiles of all units form one line that is cut into equal pieces,
// one per CTA of a single wave, whatever the mix of lengths (the lengths are on
// the device; every CTA sums them itself).  A unit that is cut leaves partial
// sums in a workspace, which a second, programmatically dependent kernel joins.
//
// Measured (6792 GB/s is a plain copy): 256 slots, 32 x 8 heads of 128, contexts
// up to 8192, e4m3: 360 us, 6.4 TB/s (float32 queries 398 us); 64 slots, 16 x 2
// heads of 256, int8: 67 us, 4.6 TB/s, of which 15 us are the start, the units'
// starts and the join (float32 77 us).  With registers as the stages (no rings)
// the first took 395 us and the second 77.  d = 64 reaches 3.3 (int8) and 3.9
// TB/s (e4m3): there a step's fixed instructions outweigh its bytes.  Float32
// prompts run here too, 16 rows at a time: 2048 tokens of 32 x 8 x 128 take 472
// us, 8192 take 6.4 ms, 86 TFLOP/s.
#include <cuda.h>

#include "gdn_kv.cuh"
#include "gdn_kv_cut.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16 * kWarps;      // tokens
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 7.f, kLift = 8.f;
constexpr int kHigh = 50;  // V exponents of ordinary pages: from kHigh - kFar up to this

// A unit that is cut starts in CTA c and ends in CTA c + parts - 1 (parts 0: none does).
struct CutUnit {
  int parts, tok0, head, row0, rows, pad[3];
};

template <int D, int NT, int PARTS>
struct SplitCfg {
  static constexpr int kRows = 8 * NT;
  // CTAs per SM that the register budget is set for
  static constexpr int kCtas = D == 64 ? (NT == 1 ? 5 : 4) : D == 128 ? (NT == 1 ? 4 : 3)
                                                                      : (NT == 1 ? 3 : 2);
  // What a unit's start costs a CTA (its queries, its first page ids and codes), in tiles:
  // the line of tiles is cut as if each unit had so many more (where there are many tiles per
  // CTA; else every CTA should have as few as possible).  Measured on 64 contexts up to 8192,
  // d = 256: a second unit takes a CTA 5 us, a tile 2.4 us; for the other d the same bytes, not
  // measured.
  static constexpr int kEntry = 512 / D;
  // Shares of an SM's CTAs.  The warps that came first are issued first: with equal shares
  // the three CTAs of d = 256 (NT = 1) end after 44, 47.5 and 53 us.
  static constexpr int kShare(int order) { return D == 256 && NT == 1 ? 13 - order : 1; }
  static constexpr int kSkewed = D == 256 && NT == 1;
  // stages of a warp's ring: what fits in an SM's shared memory with kCtas CTAs
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? (NT == 1 ? 3 : 4)
                                                        : (NT == 1 ? 2 : PARTS == 1 ? 3 : 2);
  static constexpr int kStage = 2 * 16 * D;            // bytes: K, then V
  static constexpr int kPartFloats = kRows * (D + 2);  // O, then M, then L
  static constexpr int kOutStride = D + 4;             // floats; spreads the rows over the banks
  // the rings, and after the last tile the warps' sums in their place
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSums = kWarps * kRows * kOutStride * 4;
  static constexpr int kSmem = (kRing > kSums ? kRing : kSums) + PARTS * kRows * D * 2 + 1024;
};

// What one sequence asks for.
struct SeqWork {
  int slot, tok0, len, kv_len;
  int row_tiles, tiles;   // row tiles per KV head; token tiles per unit
  int64_t weight;         // length of all its units; 0: nothing (or a bad entry)
};

__device__ __forceinline__ SeqWork seq_work(const KVView &c, const KVAttendArgs &a, int i,
                                            int rows_per_unit, int entry, bool report) {
  SeqWork w;
  w.weight = 0;
  w.slot = a.seq.slot_ids[i];
  w.kv_len = a.kv_lens[i];
  w.tok0 = i;
  int hi = i + 1;
  if (a.seq.cu_seqlens != nullptr) {
    w.tok0 = a.seq.cu_seqlens[i];
    hi = a.seq.cu_seqlens[i + 1];
  }
  w.len = hi - w.tok0;
  if (w.slot < 0 || w.slot >= c.n_slots) {
    if (report) raise_error(c.err, GDN_DEVERR_SLOT);
    return w;
  }
  if (w.tok0 < 0 || hi < w.tok0 || hi > a.seq.total_tokens || w.kv_len < 0 ||
      w.kv_len > c.capacity()) {
    if (report) raise_error(c.err, GDN_DEVERR_SEQ);
    return w;
  }
  const int64_t rows = (int64_t)w.len * (c.h_q / c.h_kv);
  w.row_tiles = (int)((rows + rows_per_unit - 1) / rows_per_unit);
  w.tiles = w.kv_len > 0 ? (w.kv_len + kTile - 1) / kTile : 1;
  w.weight = (int64_t)c.h_kv * w.row_tiles * (w.tiles + entry);
  return w;
}

// Exclusive prefix sum over the CTA's threads, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *buf, int64_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t own = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int64_t from = x - own, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) from += buf[w];
    all += buf[w];
  }
  *total = all;
  return from;
}

__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

using kv::fast_exp2;

// 16 rows of 128 (d = 64: 64) bytes: bytes x.. of rows `row`.. of block `blk`
__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *m, int x, int row, int blk,
                                         uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(row), "r"(blk), "r"(smem_addr(bar))
      : "memory");
}

// Conversions of packed codes to binary16 pairs.  k_pairs: the four codes of a
// word as two pairs; byte b of the word is element place(b) of the four.  v_pairs: byte b of two tokens' words as pair b.
template <int CODE>
struct Pairs;

template <>
struct Pairs<GDN_KV_I8> {
  // the pairs are bytes (0, 2) and (1, 3): byte 0..3 is element 0, 2, 1, 3
  static __device__ __forceinline__ int place(int byte) { return (byte & 1) * 2 + (byte >> 1); }
  // 0x6400 | (code + 128) is 1152 + code in binary16; exact
  static __device__ __forceinline__ uint32_t widen(uint32_t bytes) {
    uint32_t x = (bytes & 0x00ff00ffu) ^ 0x64806480u, y;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x64806480u));
    return y;
  }
  static __device__ __forceinline__ void k_pairs(uint32_t w, uint32_t &p, uint32_t &q) {
    p = widen(w);
    q = widen(w >> 8);
  }
  static __device__ __forceinline__ void v_pairs(uint32_t w0, uint32_t w1, uint32_t *p) {
    const uint32_t a = __byte_perm(w0, w1, 0x5410), b = __byte_perm(w0, w1, 0x7632);
    p[0] = widen(a);
    p[1] = widen(a >> 8);
    p[2] = widen(b);
    p[3] = widen(b >> 8);
  }
};

template <>
struct Pairs<GDN_KV_E4M3> {
  static __device__ __forceinline__ int place(int byte) { return byte; }
  static __device__ __forceinline__ void split(uint32_t w, uint32_t &p, uint32_t &q) {
    p = kv::e4m3x2_to_half2((uint16_t)(w & 0xffffu));
    q = kv::e4m3x2_to_half2((uint16_t)(w >> 16));
  }
  static __device__ __forceinline__ void k_pairs(uint32_t w, uint32_t &p, uint32_t &q) {
    split(w, p, q);
  }
  static __device__ __forceinline__ void v_pairs(uint32_t w0, uint32_t w1, uint32_t *p) {
    split(__byte_perm(w0, w1, 0x5140), p[0], p[1]);
    split(__byte_perm(w0, w1, 0x7362), p[2], p[3]);
  }
};

// Token of product row (or k index) r of a 16-token step.
__device__ __forceinline__ int perm(int r) { return (r & 8) | (r & 1 ? (r & 7) ^ 4 : r & 7); }

// Byte offset of 16-byte chunk x of row `row` in a stage's K or V half, as the
// tensor copy swizzles it.
template <int D>
__device__ __forceinline__ int chunk_at(int row, int x) {
  if constexpr (D == 64) return row * 64 + ((x ^ (row >> 1 & 3)) << 4);
  return (x >> 3) * 2048 + row * 128 + (((x & 7) ^ (row & 7)) << 4);
}

// V words of token `row`: d from 16 g (+ 128 i), for D = 64 from 8 g
template <int D>
__device__ __forceinline__ void load_v(uint32_t *w, const unsigned char *v, int row, int g) {
  if constexpr (D == 64) {
    const uint2 x = *reinterpret_cast<const uint2 *>(v + chunk_at<D>(row, g >> 1) + 8 * (g & 1));
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < D / 128; ++i) {
      const uint4 x = *reinterpret_cast<const uint4 *>(v + chunk_at<D>(row, 8 * i + g));
      w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
  }
}

// d of byte 0 of word j of a lane's V words
template <int D>
__device__ __forceinline__ int v_dim(int g, int j) {
  return D == 64 ? 8 * g + 4 * j : 128 * (j / 4) + 16 * g + 4 * (j % 4);
}

__device__ __forceinline__ void put_row4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put_row4(bf16 *p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

// o = O / L of one row's four elements; a row without weights is zero
__device__ __forceinline__ void put_out(const KVView &c, const KVAttendArgs &a, int tok0, int head,
                                        int row, int d, float4 x, float l) {
  const int group = c.h_q / c.h_kv;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)(tok0 + row / group) * a.ld_o +
                     (int64_t)(head * group + row % group) * c.d + d;
  if (a.o_dtype == GDN_F32)
    put_row4(static_cast<float *>(a.o) + at, scale4(inv, x));
  else
    put_row4(static_cast<bf16 *>(a.o) + at, scale4(inv, x));
}

template <int CODE, int D, int NT, typename TQ>
__global__ void __launch_bounds__(kThreads, SplitCfg<D, NT, sizeof(TQ) == 4 ? 2 : 1>::kCtas)
    attend_split_kernel(const __grid_constant__ CUtensorMap k_map,
                        const __grid_constant__ CUtensorMap v_map, const KVView c, const int layer,
                        const KVAttendArgs a, const int entry, const bool full_grid,
                        float *__restrict__ part,
                        CutUnit *__restrict__ cut) {
  constexpr int PARTS = sizeof(TQ) == 4 ? 2 : 1;  // binary16 parts of queries and weights
  using Cfg = SplitCfg<D, NT, PARTS>;
  constexpr int R = Cfg::kRows, S = Cfg::kStages;
  constexpr int SEGS = D / 64, VW = D / 32, MT = D / 16;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *sO = reinterpret_cast<float *>(smem);  // [kWarps][R][kOutStride], after the rings
  __half *sQ = reinterpret_cast<__half *>(      // [PARTS][NT][SEGS][2][32][8]
      smem + (Cfg::kRing > Cfg::kSums ? Cfg::kRing : Cfg::kSums));
  __shared__ float sM[kWarps][R], sL[kWarps][R], sA[R];
  __shared__ int64_t s_buf[kWarps], s_found_off;
  __shared__ int s_found;
  __shared__ __align__(8) uint64_t s_full[kWarps][S];

  kv::dependents_may_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int n = a.seq.n_seqs, cta = blockIdx.x;
  const int group = c.h_q / c.h_kv;
  unsigned char *ring = smem + warp * S * Cfg::kStage;
  uint64_t *full = s_full[warp];
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&full[i], 1);
    mbar_fence_init();
    // (test hook: the first copy's barrier waits for 16 bytes that no one sends)
    if ((c.test_flags & GDN_TEST_KV_WAIT_TIMEOUT) && warp == 0 && (cta & 1))
      mbar_expect_tx(&full[0], 16);
  }

  // ---- this CTA's piece of the line of tiles ----
  if (tid == 0) s_found = -1;
  kv::dependent_wait();
  if (tid == 0) cut[cta].parts = 0;
  const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int64_t mine = 0, total;
  for (int i = i0; i < i1; ++i) mine += seq_work(c, a, i, R, entry, cta == 0).weight;
  int64_t from = block_scan(mine, s_buf, &total);
  const int ctas = (int)min(total, (int64_t)gridDim.x);
  if (cta >= ctas) return;
  // (a full grid has sm_count * kCtas CTAs; CTA i is the (i / sm_count)-th of its SM)
  const bool skewed = Cfg::kSkewed && full_grid && ctas == (int)gridDim.x && total >= 4 * ctas;
  const Cut<Cfg> cuts{total, skewed ? ctas / Cfg::kCtas : ctas, skewed ? Cfg::kCtas : 1};
  const int64_t begin = cuts.begin(cta), end = cuts.begin(cta + 1);
  if (from <= begin && begin < from + mine)
    for (int i = i0; i < i1; ++i) {
      const int64_t x = seq_work(c, a, i, R, entry, false).weight;
      if (from <= begin && begin < from + x) {
        s_found = i;
        s_found_off = begin - from;
      }
      from += x;
    }
  __syncthreads();

  int seq = s_found;
  if (seq < 0) return;  // (only if the lengths changed under the kernel)
  SeqWork w = seq_work(c, a, seq, R, entry, false);
  if (w.weight == 0) return;
  int unit, place;  // place: in the unit, its entry first
  {
    const int64_t off = s_found_off;
    const int len = w.tiles + entry;
    unit = (int)(off >> 32 == 0 ? (uint32_t)off / (uint32_t)len : off / len);
    place = (int)(off - (int64_t)unit * len);
  }
  int at_stage = 0;      // the ring's next stage, and the phase of its barrier
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t at = begin; at < end && ok;) {
    if (unit == c.h_kv * w.row_tiles) {  // the next sequence that has work
      do {
        if (++seq >= n) return;
        w = seq_work(c, a, seq, R, entry, false);
      } while (w.weight == 0);
      unit = 0;
    }
    const int64_t unit_end = at + w.tiles + entry - place;
    const int tile = max(place - entry, 0);
    const int n_here = (int)(min(unit_end, end) - at) + place - entry - tile;
    at = min(unit_end, end);
    place = 0;
    if (n_here <= 0) continue;  // the piece ends within the unit's entry
    const int head = unit / w.row_tiles, row0 = (unit % w.row_tiles) * R;
    const int rows = (int)min((int64_t)w.len * group - row0, (int64_t)R);
    const int pos0 = w.kv_len - w.len + 1;            // positions open to token 0
    const int lim_min = pos0 + row0 / group;          // ... to every row of the unit
    const int last = min((tile + n_here) * kTile, pos0 + (row0 + rows - 1) / group);
    const int32_t *table = c.table + (int64_t)w.slot * c.max_pages;
    const int tok0 = tile * kTile + 16 * warp;
    const int steps = tok0 < last ? (last - tok0 + kTile - 1) / kTile : 0;

    // A step's block of codes, or -1 (reported) if its page id is bad: block 0 is read in its
    // place, and its tokens are masked.
    const int blk0 = layer * c.n_pages * c.h_kv + head;
    auto block_of = [&](int i) {
      const int id = table[(tok0 + i * kTile) >> c.page_log2];
      return (uint32_t)id < (uint32_t)c.n_pages ? id * c.h_kv + blk0 : -1;
    };
    auto fill = [&](int i, int blk, int stage) {
      if (lane == 0) {
        if (blk < 0) raise_error(c.err, GDN_DEVERR_PAGE);
        const int row = (tok0 + i * kTile) & (c.page_tokens - 1);
        unsigned char *dst = ring + stage * Cfg::kStage;
        uint64_t *bar = &full[stage];
        mbar_arrive_expect_tx(bar, Cfg::kStage);
#pragma unroll
        for (int x = 0; x < D; x += 128) tma_rows(dst + 16 * x, &k_map, x, row, max(blk, 0), bar);
#pragma unroll
        for (int x = 0; x < D; x += 128)
          tma_rows(dst + 16 * D + 16 * x, &v_map, x, row, max(blk, 0), bar);
      }
    };
    int ids[S];
#pragma unroll
    for (int i = 0; i < S; ++i) ids[i] = i < steps ? block_of(i) : -1;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < steps) fill(i, ids[i], at_stage + i < S ? at_stage + i : at_stage + i - S);

    // ---- queries: scaled by a power of two, binary16, in the B layout ----
    constexpr int E = D / 32;
    for (int r = warp; r < R; r += kWarps) {
      const int row = row0 + min(r, rows - 1);  // rows past the end repeat the last, unused
      const TQ *q = static_cast<const TQ *>(a.q) + (int64_t)(w.tok0 + row / group) * a.ld_q +
                    (int64_t)(head * group + row % group) * D + lane * E;
      float x[E];
      if constexpr (E == 2) {
        x[0] = Elem<TQ>::load1(q);
        x[1] = Elem<TQ>::load1(q + 1);
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 f = Elem<TQ>::load4(q + e);
          x[e] = f.x, x[e + 1] = f.y, x[e + 2] = f.z, x[e + 3] = f.w;
        }
      }
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(x[e]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      int ex = (int)(__float_as_uint(m) >> 23) - 127;
      ex = kv::query_exponent(ex, m == 0.f);
      const float inv = a.scale < 0.f ? -kv::pow2f(-ex) : kv::pow2f(-ex);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int d = lane * E + e;
        const int j = (d & 12) + Pairs<CODE>::place(d & 3);  // place within the lane's 16
        const int dst = ((((r >> 3) * SEGS + d / 64) * 2 + (j >> 3)) * 32 + (r & 7) * 4 +
                         (d % 64) / 16) * 8 + (j & 7);
        const float y = x[e] * inv;
        const __half hi = __float2half_rn(y);
        sQ[dst] = hi;
        if constexpr (PARTS == 2) sQ[NT * 8 * D + dst] = __float2half_rn(y - __half2float(hi));
      }
      if (lane == 0) sA[r] = fabsf(a.scale) * kLog2e * kv::pow2f(ex);
    }
    __syncthreads();

    // ---- the tiles ----
    float o[MT][NT][4], M[NT][2], Ms[NT][2], L[NT][2], qa[NT][2];
    int lim[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        M[x][y] = -INFINITY;
        Ms[x][y] = -1e30f;  // any exponent is above it: the first positions raise M
        L[x][y] = 0.f;
        qa[x][y] = sA[8 * x + 2 * t + y];
        lim[x][y] = pos0 + (row0 + min(8 * x + 2 * t + y, rows - 1)) / group;
      }
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) o[x][y][z] = 0.f;
    uint32_t odd_low = (uint32_t)(127 + kHigh - kv::kFar) << 23;
    // scales of the next step, loaded a step ahead
    float next_k = 0.f, next_v = 0.f;
    auto scales = [&](int blk) {
      next_k = c.k_scale[max(blk, 0)];
      next_v = c.v_scale[max(blk, 0)];
    };
    if (steps > 0) scales(ids[0]);
    int ahead = S < steps ? block_of(S) : -1;  // block of step i + S
    for (int i = 0; i < steps && ok; ++i) {
      const int tok = tok0 + i * kTile, stage = at_stage;
      const unsigned char *sK = ring + stage * Cfg::kStage, *sV = sK + 16 * D;
      const bool valid = ids[0] >= 0;
      const float k_scale = next_k;
      // the V scale is 2^e: e, and 2^-e (a block that only stands in for a bad page: 1)
      const uint32_t v_bits = valid ? __float_as_uint(next_v) & 0x7f800000u : 0x3f800000u;
      const float e = (float)((int)(v_bits >> 23) - 127);
      // Exponents that lie far from the others' (see gdn_kv.cuh): none do while all are from
      // kHigh - kFar to kHigh; a larger one moves the lower end.  Their terms of L are added apart.
      const bool odd = v_bits < odd_low || v_bits > (uint32_t)(127 + kHigh) << 23;
      float unscale = __uint_as_float(0x7f000000u - v_bits);
#pragma unroll
      for (int x = 0; x + 1 < S; ++x) ids[x] = ids[x + 1];
      ids[S - 1] = ahead;
      if (i + 1 < steps) scales(ids[0]);
      if (i + S + 1 < steps) ahead = block_of(i + S + 1);
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase));
      if (++at_stage == S) {
        at_stage = 0;
        phase ^= 1;
      }
      if (!ok) {  // report it, and give the copies in flight (with limits again) time to land
        if (lane == 0) raise_error(c.err, GDN_DEVERR_TIMEOUT);
        for (int x = i + 1; x < min(steps, i + S); ++x) {
          mbar_wait_bounded(&full[at_stage], phase);
          if (++at_stage == S) {
            at_stage = 0;
            phase ^= 1;
          }
        }
        break;
      }

      // S^T = K Q^T
      float s[NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
      for (int seg = 0; seg < SEGS; ++seg) {
        // (float32 queries: the products' own sums are short, and joined by rounded additions)
        float part_s[PARTS == 2 ? NT : 1][4] = {};
        const uint4 k0 = *reinterpret_cast<const uint4 *>(sK + chunk_at<D>(perm(g), 4 * seg + t));
        const uint4 k1 =
            *reinterpret_cast<const uint4 *>(sK + chunk_at<D>(perm(g + 8), 4 * seg + t));
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
          uint32_t a0[4], a1[4];
          Pairs<CODE>::k_pairs(w0[2 * j2], a0[0], a0[2]);
          Pairs<CODE>::k_pairs(w1[2 * j2], a0[1], a0[3]);
          Pairs<CODE>::k_pairs(w0[2 * j2 + 1], a1[0], a1[2]);
          Pairs<CODE>::k_pairs(w1[2 * j2 + 1], a1[1], a1[3]);
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              const uint4 b = *reinterpret_cast<const uint4 *>(
                  sQ + (size_t)((((p * NT + x) * SEGS + seg) * 2 + j2) * 32 + lane) * 8);
              float *sum = PARTS == 2 ? part_s[x] : s[x];
              mma16816(sum, a0, b.x, b.y);
              mma16816(sum, a1, b.z, b.w);
            }
        }
        if constexpr (PARTS == 2)
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) s[x][y] += part_s[x][y];
      }
      // weights
      const bool masked = tok + 16 > lim_min || !valid;
      float f[NT][2], y[NT][4];  // y: exponents of the weights
      auto exponents = [&](int x, int k, float shift) {
        y[x][k] = fmaf(s[x][k], f[x][k], shift);
        y[x][2 + k] = fmaf(s[x][2 + k], f[x][k], shift);
        if (masked) {
          if (!valid || tok + perm(g) >= lim[x][k]) y[x][k] = -INFINITY;
          if (!valid || tok + perm(g + 8) >= lim[x][k]) y[x][2 + k] = -INFINITY;
        }
      };
      bool raise = odd;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f[x][k] = qa[x][k] * k_scale;
          exponents(x, k, e - Ms[x][k]);
          raise |= fmaxf(y[x][k], y[x][2 + k]) > kSlack + kLift;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            exponents(x, k, e);
            float m = fmaxf(y[x][k], y[x][2 + k]) + fmaxf(kv::kLowExp - e, 0.f);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            m = fmaxf(ceilf(m), M[x][k]);
            if (m != -INFINITY) {
              const float keep = fast_exp2(M[x][k] - m);
              L[x][k] = kv::lower(L[x][k], M[x][k] - m);
              M[x][k] = m;
              Ms[x][k] = m - kLift;
#pragma unroll
              for (int j = 0; j < MT; ++j) {
                o[j][x][k] *= keep;
                o[j][x][2 + k] *= keep;
              }
            }
            exponents(x, k, e - Ms[x][k]);
            if (odd) {
#pragma unroll
              for (int z = k; z < 4; z += 2)
                if (y[x][z] != -INFINITY)
                  L[x][k] += kv::lower(1.f, fmaf(s[x][z], f[x][k], -Ms[x][k]));
            }
          }
        if (odd) unscale = 0.f;
        constexpr uint32_t kSpan = (uint32_t)kv::kFar << 23;
        odd_low = max(odd_low, max(v_bits, kSpan) - kSpan);
      }
      uint32_t pb[PARTS][NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = fast_exp2(y[x][k]);
        L[x][0] = fmaf(p[0] + p[2], unscale, L[x][0]);
        L[x][1] = fmaf(p[1] + p[3], unscale, L[x][1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t h = half2_bits(p[2 * k], p[2 * k + 1]);
          pb[0][x][k] = transpose8(h);
          if constexpr (PARTS == 2) {
            const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            pb[1][x][k] = transpose8(half2_bits(p[2 * k] - r.x, p[2 * k + 1] - r.y));
          }
        }
      }

      // O^T += V^T P^T
      uint32_t vw[4][VW];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        load_v<D>(vw[x], sV, perm(2 * t + (x & 1) + 8 * (x >> 1)), g);
      if (tok + 16 > w.kv_len || !valid) {  // what lies there is no code of this sequence
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (!valid || tok + perm(2 * t + (x & 1) + 8 * (x >> 1)) >= w.kv_len)
#pragma unroll
            for (int j = 0; j < VW; ++j) vw[x][j] = 0;
      }
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        uint32_t lo[4], hi[4];
        Pairs<CODE>::v_pairs(vw[0][j], vw[1][j], lo);
        Pairs<CODE>::v_pairs(vw[2][j], vw[3][j], hi);
        const uint32_t a0[4] = {lo[0], lo[1], hi[0], hi[1]};
        const uint32_t a1[4] = {lo[2], lo[3], hi[2], hi[3]};
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          if constexpr (PARTS == 1) {
            mma16816(o[2 * j][x], a0, pb[0][x][0], pb[0][x][1]);
            mma16816(o[2 * j + 1][x], a1, pb[0][x][0], pb[0][x][1]);
          } else {
            float u[4] = {}, v[4] = {};
            mma16816(u, a0, pb[1][x][0], pb[1][x][1]);
            mma16816(v, a1, pb[1][x][0], pb[1][x][1]);
            mma16816(u, a0, pb[0][x][0], pb[0][x][1]);
            mma16816(v, a1, pb[0][x][0], pb[0][x][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              o[2 * j][x][k] += u[k];
              o[2 * j + 1][x][k] += v[k];
            }
          }
        }
      }
      __syncwarp();  // the stage has been read by every lane
      if (i + S < steps) fill(i + S, ids[S - 1], stage);
    }
    // the rings are free after this: the sums take their place
    ok = __syncthreads_and(ok);

    // ---- join the warps ----
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float l = L[x][y];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int r = 8 * x + 2 * t + y;
        if (g == 0) {
          sM[warp][r] = ok ? M[x][y] : kv::no_result();  // (of every warp: the join finds it)
          sL[warp][r] = l;
        }
#pragma unroll
        for (int j = 0; j < VW; ++j)
          *reinterpret_cast<float4 *>(sO + (size_t)(warp * R + r) * Cfg::kOutStride +
                                      v_dim<D>(g, j)) =
              make_float4(o[2 * j][x][y], o[2 * j][x][2 + y], o[2 * j + 1][x][y],
                          o[2 * j + 1][x][2 + y]);
      }
    __syncthreads();
    const bool whole = n_here == w.tiles;
    float *my_part = part + (size_t)(2 * cta + (tile == 0 ? 1 : 0)) * Cfg::kPartFloats;
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = 4 * (x % (D / 4));
      float m = sM[0][r];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) m = fmaxf(m, sM[k][r]);
      float l = 0.f;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float f = kv::join_factor(sL[k][r], sM[k][r], m);
        l += kv::join_sum(sL[k][r], sM[k][r], m);
        sum = axpby4(1.f, sum, f,
                     *reinterpret_cast<const float4 *>(sO + (size_t)(k * R + r) * Cfg::kOutStride +
                                                       d));
      }
      if (whole) {
        if (ok) put_out(c, a, w.tok0, head, row0 + r, d, sum, l);
      } else {
        *reinterpret_cast<float4 *>(my_part + r * D + d) = sum;
        if (d == 0) {
          my_part[R * D + r] = m;
          my_part[R * D + R + r] = l;
        }
      }
    }
    if (tid == 0 && !whole && tile == 0)
      cut[cta] = CutUnit{cuts.owner(unit_end - 1) - cta + 1, w.tok0, head, row0, rows, {0, 0, 0}};
    // the next unit's copies (async proxy) overwrite what was written here
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    ++unit;
  }
}

// Joins the parts of the unit that was cut at the end of CTA blockIdx.x, one
// query row per CTA.  Maxima and sums of all parts, and the first outputs, are
// loaded at once: what counts is how few loads wait for one another.
constexpr int kJoinThreads = 256;
constexpr int kMaxGrid = 2048;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads)
    attend_join_kernel(const KVView c, const KVAttendArgs a, const float *part,
                       const CutUnit *cut) {
  using Cfg = SplitCfg<D, NT, 1>;
  constexpr int R = Cfg::kRows;
  constexpr int COLS = D / 4;                   // float4 columns of a row
  constexpr int ACROSS = kJoinThreads / COLS;   // threads of a column share the parts
  constexpr int FIRST = 4;                      // outputs that a thread loads ahead
  __shared__ float4 s_sum[kJoinThreads];
  __shared__ float s_f[kMaxGrid], s_red[2][kJoinThreads / 32];
  // (No early launch of what follows: a next attention call, resident while this grid is still
  // being worked off, ends later.  256 contexts, call after call: 433 us with it, 364 without;
  // drafts of d = 256: 126 and 128.)
  kv::dependent_wait();
  const CutUnit u = cut[blockIdx.x];
  const int r = blockIdx.y;
  if (u.parts == 0 || r >= u.rows) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int col = tid % COLS, share = tid / COLS;
  // part 0 is the second partial sum of CTA blockIdx.x, part p the first of CTA blockIdx.x + p
  auto at = [&](int p) {
    return part + (size_t)(2 * (blockIdx.x + p) + (p == 0 ? 1 : 0)) * Cfg::kPartFloats;
  };
  auto out = [&](int p) {
    return __ldcg(reinterpret_cast<const float4 *>(at(p) + r * D + 4 * col));
  };
  float4 first[FIRST];
#pragma unroll
  for (int x = 0; x < FIRST; ++x)
    if (share + x * ACROSS < u.parts) first[x] = out(share + x * ACROSS);
  float m = -INFINITY, own_m = -INFINITY, own_l = 0.f;
  bool missing = false;
  for (int p = tid; p < u.parts; p += kJoinThreads) {
    own_m = __ldcg(at(p) + R * D + r);
    own_l = __ldcg(at(p) + R * D + R + r);
    s_f[p] = own_m;
    missing |= own_m != own_m;
    m = fmaxf(m, own_m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  missing = __any_sync(0xffffffffu, missing);
  if (lane == 0) s_red[0][warp] = missing ? kv::no_result() : m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinThreads / 32; ++k) {
    missing |= s_red[0][k] != s_red[0][k];
    m = fmaxf(m, s_red[0][k]);
  }
  float l = 0.f;
  for (int p = tid; p < u.parts; p += kJoinThreads) {
    const float pm = s_f[p];
    const float pl = u.parts <= kJoinThreads ? own_l : __ldcg(at(p) + R * D + R + r);
    s_f[p] = kv::join_factor(pl, pm, m);
    l += kv::join_sum(pl, pm, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_red[1][warp] = l;
  __syncthreads();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int x = 0; x < FIRST; ++x)
    if (share + x * ACROSS < u.parts) sum = axpby4(1.f, sum, s_f[share + x * ACROSS], first[x]);
#pragma unroll 8
  for (int p = share + FIRST * ACROSS; p < u.parts; p += ACROSS)
    sum = axpby4(1.f, sum, s_f[p], out(p));
  s_sum[tid] = sum;
  __syncthreads();
  if (share == 0 && !missing) {  // (where some part gave up the row stays as it was)
#pragma unroll
    for (int k = 1; k < ACROSS; ++k) sum = axpby4(1.f, sum, 1.f, s_sum[k * COLS + col]);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinThreads / 32; ++k) l += s_red[1][k];
    put_out(c, a, u.tok0, u.head, u.row0 + r, 4 * col, sum, l);
  }
}

template <int CODE, int D, int NT, typename TQ>
cudaError_t launch_split(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                         cudaStream_t s) {
  using Cfg = SplitCfg<D, NT, sizeof(TQ) == 4 ? 2 : 1>;
  auto kernel = attend_split_kernel<CODE, D, NT, TQ>;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = kv::allow_smem(kernel, Cfg::kSmem, h.device, seen);
  if (e != cudaSuccess) return e;
  // one wave, or fewer CTAs where the hints say that there are fewer tiles
  const int64_t rows = (int64_t)a.max_seqlen * (c.h_q / c.h_kv);
  const double tiles = (double)a.seq.n_seqs * c.h_kv * ((rows + Cfg::kRows - 1) / Cfg::kRows) *
                       (a.max_kv_len / kTile + 1);
  const int64_t most = (int64_t)h.sm_count * Cfg::kCtas;
  // A CTA per tile where there are fewer tiles than that; two tiles where a context has more
  // than 64, as its join would get long (1 x 2 heads, 8192 tokens: 15.1 us with one tile a CTA,
  // 13.1 with two, 14.2 with three; 777 tokens: 9.5, 13.9, 14.6).
  const int least = a.max_kv_len > 64 * kTile ? 2 : 1;
  const int64_t full = most < kMaxGrid ? most : kMaxGrid;
  const int64_t grid = tiles < (double)full * least ? ((int64_t)tiles + least - 1) / least : full;
  const int entry = tiles >= 8. * (double)most ? Cfg::kEntry : 0;
  const size_t part_bytes = (size_t)grid * 2 * Cfg::kPartFloats * sizeof(float);
  void *work = nullptr;
  bool temporary;
  e = h.work->get(part_bytes + grid * sizeof(CutUnit), s, &work, &temporary);
  if (e != cudaSuccess) return e;
  float *part = static_cast<float *>(work);
  CutUnit *cut = reinterpret_cast<CutUnit *>(static_cast<char *>(work) + part_bytes);
  e = kv::launch(kernel, dim3((unsigned)grid), kThreads, Cfg::kSmem, s, 1, *h.k_map, *h.v_map, c,
                 layer, a, entry, grid == most, part, cut);
  // (one token per slot: a unit has exactly the rows of its group)
  const unsigned used = a.seq.cu_seqlens == nullptr && c.h_q / c.h_kv < Cfg::kRows
                            ? (unsigned)(c.h_q / c.h_kv)
                            : (unsigned)Cfg::kRows;
  if (e == cudaSuccess)
    e = kv::launch(attend_join_kernel<D, NT>, dim3((unsigned)grid, used), kJoinThreads, 0, s, 1, c,
                   a, static_cast<const float *>(part), static_cast<const CutUnit *>(cut));
  const cudaError_t ef = temporary ? cudaFreeAsync(work, s) : cudaSuccess;
  return e != cudaSuccess ? e : ef;
}

template <int CODE, int D, int NT>
cudaError_t by_type(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                    cudaStream_t s) {
  return a.q_dtype == GDN_F32 ? launch_split<CODE, D, NT, float>(c, layer, a, h, s)
                              : launch_split<CODE, D, NT, bf16>(c, layer, a, h, s);
}

template <int CODE, int D>
cudaError_t by_rows(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                    cudaStream_t s) {
  // eight query rows per unit where a slot has no more, else sixteen
  return (int64_t)a.max_seqlen * (c.h_q / c.h_kv) <= 8
             ? by_type<CODE, D, 1>(c, layer, a, h, s)
             : by_type<CODE, D, 2>(c, layer, a, h, s);
}

template <int CODE>
cudaError_t by_dim(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                   cudaStream_t s) {
  return c.d == 64    ? by_rows<CODE, 64>(c, layer, a, h, s)
         : c.d == 128 ? by_rows<CODE, 128>(c, layer, a, h, s)
                      : by_rows<CODE, 256>(c, layer, a, h, s);
}

}  // namespace

cudaError_t launch_kv_attend(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                             cudaStream_t s) {
  // The tcgen05 kernel takes bf16 calls with more than 16 query rows per KV head, but not the
  // small ones (its units take longer to set up) and, up to 32 rows, neither those with few
  // units, which it cannot spread as well, nor those with more than a wave of them, of whose
  // 128-row tiles it uses a quarter.  Measured, split / tcgen05 in us, as sequences x KV heads,
  // rows, context:
  //   2 x 136 x 512 15 / 23     8 x 36 x 2048 20 / 20      8 x 72 x 2048 30 / 27
  //   8 x 132 x 2048 30 / 26    16 x 264 x 2048 76 / 39    64 x 68 x 8192 161 / 70
  //   2 x 24 x 8192 22 / 29     32 x 27 x 2048 27 / 19     64 x 20 x 2048 34 / 28
  //   128 x 24 x 8192 212 / 222   192 x 20 x 2048 67 / 77  512 x 20 x 512 56 / 73
  const int64_t rows = (int64_t)a.max_seqlen * (c.h_q / c.h_kv);
  const int64_t heads = (int64_t)a.seq.n_seqs * c.h_kv;
  if (a.q_dtype == GDN_BF16 && (rows > 32 || (rows > 16 && heads >= 16 && heads <= h.sm_count)) &&
      (double)heads * ((rows + 15) / 16) * a.kv_hint > 32768.)
    return launch_kv_attend_prompt(c, layer, a, h, s);
  return c.code == GDN_KV_I8 ? by_dim<GDN_KV_I8>(c, layer, a, h, s)
                             : by_dim<GDN_KV_E4M3>(c, layer, a, h, s);
}

}  // namespace gdn
