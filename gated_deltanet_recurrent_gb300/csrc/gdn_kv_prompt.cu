// Causal grouped-query attention over the 8-bit KV cache on the 5th-generation
// tensor cores: bf16 calls with many query rows per KV head (prompts, and
// drafts of wide groups).  Mathematics, scaling and masking are those of
// gdn_kv_attend.cu; this file is about feeding tcgen05.
//
// A unit is 128 * MT query rows (token-major, the query heads of one KV head
// side by side) of one sequence and KV head; KV tiles have 128 tokens.  Per
// tile and 128 rows: S = Q K^T (128 x 128, operands in shared memory), softmax
// weights P back into S's TMEM columns as binary16, O += P V (P from TMEM, V in
// shared memory as an MN-major operand, so it needs no transposition).
//
// Roles, joined by mbarriers:
//   softmax    4 * MT warps, one thread per query row: S from TMEM, running
//              maximum and sum, P to TMEM; raises the maximum (and rescales O in
//              TMEM) only when it must, which after a few tiles is rare
//   converters CW warps: 16 codes per load, to binary16 (exact), into a ring of
//              slots in the 128-byte swizzle, K and V slots in the order of the
//              MMAs, in two teams that take turns
//   MMA        one warp, one elected lane issues; MT = 2: the two row tiles alternate, so one's softmax
//              runs under the other's products; MT = 1: S is double-buffered
//              and S of the next tile is computed under the softmax of this one
//   pages      one warp: page ids and scales of the coming tiles
//
// What bounds it: per tile and 128 rows the tensor pipe needs d * 8 cycles (4096
// products a cycle).  Shared memory (128 bytes a cycle) needs d * 6 for the
// operands, d * 4 / MT for the converted codes' writes and d * 2 / MT for their
// loads through L1: alone, more than the tensor pipe.  So long prompts run in
// pairs of CTAs (cta_group::2, 256-row products): each CTA converts and holds
// half of every K and V operand, which halves all but the queries' part (8 pieces
// of up to 2048 tokens, 16 x 2 heads, d = 256: 1422 -> 969 us when this came).
// MT = 2 halves the conversion per row; d = 256 has room in TMEM (O 256 columns,
// two S) for MT = 1 only.  Measured: those pieces 619 us (1230 TFLOP/s, tensor
// pipe 52 % active); a prompt of 8192, 32 x 8 heads, d = 128, 483 us (1140
// TFLOP/s, 48 %).  What is left is the softmax's latency between the two
// products of a tile (1550 of 3300 cycles), and 6 us of setup per unit.  d = 64
// has half the products for the same softmax: a prompt of 8192, 32 x 8 heads,
// 501 us in int8, 470 in e4m3 (550 and 585 TFLOP/s), although the e4m3 form
// spills 0.4 KB a thread.
#include <cuda.h>

#include <type_traits>

#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kBN = 128;                 // tokens of a KV tile
constexpr int kGroups = kBN / 16;        // page-aligned token groups of a tile
constexpr int kInfo = 8;                 // tiles of page info in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 7.f, kLift = 8.f;

template <int D, int MT, bool PAIR>
struct PromptCfg {
  static constexpr int kCtas = PAIR ? 2 : 1;            // that share a unit
  static constexpr int kRows = 128 * MT * kCtas;        // of a unit
  // A slot holds a K or V tile's codes for one MMA group: alone, 128 tokens x min(d, 128); in
  // a pair, this CTA's half of the operand, 64 tokens x d of K or 128 tokens x d / 2 of V.
  static constexpr int DC = D < 128 ? D : 128;
  static constexpr int kHalves = PAIR ? 1 : D / DC;     // slots of a K or V tile
  static constexpr int kSlot = PAIR ? 128 * D : kBN * DC * 2;  // bytes
  static constexpr int kKPanel = PAIR ? 8192 : 16384;   // bytes of a slot's 64 d (K), 64 d (V)
  static constexpr int kSlots = PAIR && D == 128 ? 6 : 4;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kConvWarps = MT == 2 ? 4 : 8;
  // Teams take the slots in turn, each loading its next slot's codes as soon as it has
  // converted one.  Two teams with one slot ahead: 707 us for 8 prompt pieces (d = 256) and
  // 482 for a prompt of 8192 (d = 128); one team 888 and 500, four teams 886 and 571; with two
  // slots ahead the codes do not fit in the registers (815, 672).
  static constexpr int kConvTeams = 2;
  static constexpr int kThreads = 512;  // warps 12..15: MMA, pages, two idle
  // registers per thread of each role; with 512 threads a launch has 128 each, and the
  // shares' sum may not exceed that: MT = 2: 256 * 168 + 128 * 112 + 128 * 64 = 65,536;
  // MT = 1: 128 * 184 + 256 * 112 + 128 * 64 = 60,416
  static constexpr int kSoftRegs = MT == 2 ? 168 : 184;
  static constexpr int kConvRegs = 112;
  static constexpr int kMiscRegs = 64;
  static constexpr int kSmem = MT * kQTile + kSlots * kSlot + 1024;
  // TMEM columns: S (MT tiles, or two buffers), then O
  static constexpr int kO = 2 * kBN;
  static constexpr int kTmem = 512;
  static constexpr int kPartFloats = kRows * (D + 2);
};

struct Unit {
  int slot, tok0, len, kv_len, head, row0, rows;
  int tiles, begin, end;  // KV tiles in all, and this split's
};

// f16 operands, f32 accumulator; B MN-major if `mn`
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// ---- what differs between a CTA alone and a pair (cluster of two, cta_group::2) ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on CTA 0's barrier of the pair.  What the arrival stands for lies in this CTA's
// own shared memory or TMEM and is complete before it (proxy fence, or the wait for TMEM
// stores), so the default scope will do: a cluster-scope release also waits for the
// global loads in flight, 1000 cycles for each slot.
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  else
    tc::mma_ss_f16(d, a, b, id, accumulate);
}
template <bool PAIR>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate)
        : "memory");
  else
    tc::mma_ts_f16(d, a, b, id, accumulate);
}
// arrive on `bar` (of both CTAs of a pair) when the MMAs issued so far are done
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    tc::mma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tc::tmem_alloc(slot, cols);
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                 : "memory");
  else
    tc::tmem_dealloc(taddr, cols);
}

// Shared-memory operands in the 128-byte swizzle: 128-byte rows of 64 elements,
// 8-row atoms (SBO 1024).  K-major (K and Q: rows are tokens or queries) or
// MN-major (V: rows are tokens, the K index; panels of 64 d are 16 KiB apart,
// LBO).  The low word takes the address; steps add to it.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t lbo) {
  return saddr >> 4 | (lbo >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc(uint32_t low) {
  return (uint64_t)kDescHigh << 32 | low;
}

using kv::fast_exp2;

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// (a0, a1) * b + c and (a0, a1) + (b0, b1) on register pairs
__device__ __forceinline__ float2 fma2(float2 a, float b, float c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\t"
      "mov.b64 z, {%5, %5};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// one lane of the warp (all 32 call it), in a form that keeps the warp's code uniform
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 columns of this thread's TMEM lane; the caller waits
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Four codes of a word as two binary16 pairs.  Along d, element j of four sits
// at place(j); queries are laid out the same way and outputs are read back so.
template <int CODE>
struct Widen;
template <>
struct Widen<GDN_KV_I8> {
  static __host__ __device__ constexpr int place(int j) { return (j & 1) * 2 + (j >> 1); }
  static __device__ __forceinline__ uint32_t one(uint32_t bytes) {
    uint32_t y;
    asm("sub.rn.f16x2 %0, %1, %2;"
        : "=r"(y)
        : "r"((bytes & 0x00ff00ffu) ^ 0x64806480u), "r"(0x64806480u));
    return y;
  }
  static __device__ __forceinline__ void four(uint32_t w, uint32_t &a, uint32_t &b) {
    a = one(w);
    b = one(w >> 8);
  }
};
template <>
struct Widen<GDN_KV_E4M3> {
  static __host__ __device__ constexpr int place(int j) { return j; }
  static __device__ __forceinline__ void four(uint32_t w, uint32_t &a, uint32_t &b) {
    a = kv::e4m3x2_to_half2((uint16_t)(w & 0xffffu));
    b = kv::e4m3x2_to_half2((uint16_t)(w >> 16));
  }
};

// Unit `u` (row tile, from the heaviest) of sequence i and KV head `head`, and
// the tiles of split `split` of `splits`.  False: there is none.
__device__ __forceinline__ bool find_unit(const KVView &c, const KVAttendArgs &a, int i, int head,
                                          int64_t u, int rows_per_unit, int split, int splits,
                                          bool report, Unit *w) {
  const int group = c.h_q / c.h_kv;
  w->slot = a.seq.slot_ids[i];
  w->kv_len = a.kv_lens[i];
  w->tok0 = i;
  int hi = i + 1;
  if (a.seq.cu_seqlens != nullptr) {
    w->tok0 = a.seq.cu_seqlens[i];
    hi = a.seq.cu_seqlens[i + 1];
  }
  w->len = hi - w->tok0;
  if (w->slot < 0 || w->slot >= c.n_slots) {
    if (report) raise_error(c.err, GDN_DEVERR_SLOT);
    return false;
  }
  if (w->tok0 < 0 || hi < w->tok0 || hi > a.seq.total_tokens || w->kv_len < 0 ||
      w->kv_len > c.capacity()) {
    if (report) raise_error(c.err, GDN_DEVERR_SEQ);
    return false;
  }
  const int64_t all = (int64_t)w->len * group;
  const int64_t units = (all + rows_per_unit - 1) / rows_per_unit;
  if (u >= units) return false;
  w->head = head;
  w->row0 = (int)((units - 1 - u) * rows_per_unit);
  w->rows = (int)min(all - w->row0, (int64_t)rows_per_unit);
  const int lim = w->kv_len - w->len + 1 + (w->row0 + w->rows - 1) / group;
  w->tiles = lim > 0 ? (lim + kBN - 1) / kBN : 0;
  w->begin = (int)((int64_t)w->tiles * split / splits);
  w->end = (int)((int64_t)w->tiles * (split + 1) / splits);
  return true;
}

__device__ __forceinline__ void put8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void put8(bf16 *p, const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t *>(&b);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A row's part of a tile with V exponents far from the others (see gdn_kv.cuh): the sum of its
// weights, in units of the denominator, from x - M itself; and the largest exponent, with no V
// exponent below kLowExp.  A function of its own, and reached from where the maximum is raised: 8
// prompt pieces (d = 256) take 612 us, a prompt of 8192 (d = 128) 490; inlined there 640 and 481,
// before the common pass over S 652 and 528.
__device__ __noinline__ float2 weigh_apart(uint32_t tS, int open, float qa, float Ms,
                                           const float *ks, const float *ve) {
  float sum = 0.f, peak = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < kBN; h += 32) {
    uint32_t v[32];
    tmem_ld32_async(tS + h, v);
    tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 32; ++x) {
      const float e = ve[(h + x) / 16];
      if (h + x < open && e != -INFINITY) {
        const float z = fmaf(__uint_as_float(v[x]), qa * ks[(h + x) / 16], -Ms);
        sum += kv::lower(1.f, z);
        peak = fmaxf(peak, z + fmaxf(e, (float)kv::kLowExp));
      }
    }
  }
  return make_float2(sum, peak);
}

template <int CODE, int D, int MT, bool PAIR>
__global__ void __launch_bounds__(PromptCfg<D, MT, PAIR>::kThreads, 1)
    attend_prompt_kernel(const KVView c, const int layer, const KVAttendArgs a, const int splits,
                         const int hinted_units, const int *order, float *__restrict__ part) {
  using Cfg = PromptCfg<D, MT, PAIR>;
  constexpr int R = Cfg::kRows, NS = Cfg::kSlots, H = Cfg::kHalves, CW = Cfg::kConvWarps;
  constexpr int TEAMS = Cfg::kConvTeams;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *sQ = smem;                             // [MT][D / 64][128 rows][128 bytes]
  unsigned char *sKV = smem + MT * Cfg::kQTile;         // [NS] slots, 128-byte rows of 64 d
  __shared__ __align__(8) uint64_t slot_full[NS], slot_empty[NS], info_full[kInfo],
      info_empty[kInfo], s_full[2], p_full[MT], pv_done[MT], q_full, drain;
  __shared__ int s_blk[kInfo][kGroups], s_plain[kInfo], s_odd[kInfo];
  __shared__ float s_ks[kInfo][kGroups], s_ve[kInfo][kGroups], s_un[kInfo][kGroups];
  __shared__ uint32_t tmem_slot;
  __shared__ int s_abort;

  kv::dependents_may_launch();
  kv::dependent_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // blocks take the units of the list, or else by row tile, the heaviest of every sequence and
  // head first
  const int block = blockIdx.x / Cfg::kCtas, rank = PAIR ? (int)cluster_rank() : 0;
  const int place0 = order ? __ldcg(order + block) : block;
  const int heads = a.seq.n_seqs * c.h_kv, z = place0 % heads, split = blockIdx.y;
  const int i = z / c.h_kv, head = z % c.h_kv, group = c.h_q / c.h_kv;
  const int64_t u0 = place0 / heads;
  Unit w;
  if (!find_unit(c, a, i, head, u0, R, 0, 1, tid + split + rank + (int)u0 == 0, &w)) return;
  constexpr int kConv = 4 * MT, kMma = kConv + CW, kPages = kMma + 1;
  static_assert(TEAMS <= NS, "a team's wait for a free slot counts on the earlier teams' slots");
  static_assert(kMma == 12, "four warpgroups: softmax and converters, then MMA and pages");
  if (tid == 0) {
    // (test hook: the first slot waits for an arrival that never comes)
    const int extra =
        (c.test_flags & GDN_TEST_KV_WAIT_TIMEOUT) && ((block + blockIdx.y) & 1) ? 1 : 0;
    for (int i = 0; i < NS; ++i)
      mbar_init(&slot_full[i], CW / TEAMS * Cfg::kCtas + (i == 0 ? extra : 0)),
          mbar_init(&slot_empty[i], 1);
    for (int i = 0; i < kInfo; ++i)
      mbar_init(&info_full[i], 1),
          mbar_init(&info_empty[i], 2 * H * (CW / TEAMS) + 4 * MT);  // its slots' loads, softmax
    for (int i = 0; i < 2; ++i) mbar_init(&s_full[i], 1);
    for (int i = 0; i < MT; ++i) mbar_init(&p_full[i], 4 * Cfg::kCtas), mbar_init(&pv_done[i], 1);
    mbar_init(&q_full, 4 * MT * Cfg::kCtas);
    mbar_init(&drain, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == kMma) tmem_alloc<PAIR>(&tmem_slot, Cfg::kTmem);
  tc::fence_before_sync();
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;
  volatile int *abort_flag = &s_abort;
  // A wait that gives up ends the kernel's work: every role stops at its next wait.
  auto wait = [&](uint64_t *bar, uint32_t phase) {
    if (mbar_wait_bounded(bar, phase & 1) && !*abort_flag) return true;
    if (*abort_flag == 0) raise_error(c.err, GDN_DEVERR_TIMEOUT);
    *abort_flag = 1;
    return false;
  };
  // slot_full, q_full and p_full are waited for by the MMA warp, which is CTA 0's in a pair
  auto arrive_mma = [&](uint64_t *bar) {
    if constexpr (PAIR)
      arrive_leader(bar);
    else
      mbar_arrive(bar);
  };
  auto warp_wait = [&](uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait(bar, phase));
  };

  uint32_t slots = 0;  // slots used by earlier units
  uint32_t done = 0;   // tiles of earlier units
  uint32_t units = 0;  // earlier units with tiles
  bool ok = true;
  // Every role walks the same units: one, or, where there are more than the
  // hint says, several, of which the later ones are not split.
  auto each_unit = [&](auto role) {
    for (int64_t u = u0; ok && find_unit(c, a, i, head, u, R, u < hinted_units ? split : 0,
                                         u < hinted_units ? splits : 1, false, &w);
         u += hinted_units) {
      if (u >= hinted_units && split > 0) break;
      const int T = w.end - w.begin;
      role(u, T);
      slots += 2 * H * T;
      done += T;
      units += T > 0;
    }
  };

  if (warp < kConv) {
    set_regs_up<Cfg::kSoftRegs>();
    each_unit([&](const int64_t u, const int T) {
      // ---- softmax: one thread per query row ----
      const int mt = warp >> 2;
      const int tile_row = 128 * (mt * Cfg::kCtas + rank) + 32 * (warp & 3);
      const int row = tile_row + lane;                    // in the unit
      const int grow = w.row0 + min(row, w.rows - 1);     // rows past the end repeat the last
      const int lim = w.kv_len - w.len + 1 + grow / group;
      float qa = 0.f;  // scale * log2(e) * the query's power of two
      if (T > 0) {
        // a lane takes E consecutive elements of each row; the next eight rows are on their
        // way while eight are scaled and stored
        constexpr int E = D / 32, kBatch = 8;
        const int row_w = w.row0 + tile_row, last_row = w.row0 + w.rows - 1;
        uint32_t raw[2][kBatch][E / 2];
        auto load_rows = [&](int r0, uint32_t (*x)[E / 2]) {
#pragma unroll
          for (int r = 0; r < kBatch; ++r) {
            const int gr = min(row_w + r0 + r, last_row);
            const bf16 *q = static_cast<const bf16 *>(a.q) +
                            (int64_t)(w.tok0 + gr / group) * a.ld_q +
                            (int64_t)(head * group + gr % group) * D + lane * E;
            if constexpr (E == 8) {
              const uint4 v = *reinterpret_cast<const uint4 *>(q);
              x[r][0] = v.x, x[r][1] = v.y, x[r][2] = v.z, x[r][3] = v.w;
            } else if constexpr (E == 4) {
              const uint2 v = *reinterpret_cast<const uint2 *>(q);
              x[r][0] = v.x, x[r][1] = v.y;
            } else {
              x[r][0] = *reinterpret_cast<const uint32_t *>(q);
            }
          }
        };
        load_rows(0, raw[0]);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += kBatch) {
          if (r0 + kBatch < 32) load_rows(r0 + kBatch, raw[(r0 / kBatch + 1) & 1]);
#pragma unroll
          for (int r = 0; r < kBatch; ++r) {
            const uint32_t *x = raw[(r0 / kBatch) & 1][r];
            uint32_t m = 0;  // magnitudes of bf16 order like their bits; NaN is left out
            float f[E];
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              f[e] = __uint_as_float(x[e / 2] << 16);
              f[e + 1] = __uint_as_float(x[e / 2] & 0xffff0000u);
              const uint32_t lo = __float_as_uint(f[e]) & 0x7fffffffu;
              const uint32_t hi = __float_as_uint(f[e + 1]) & 0x7fffffffu;
              if (lo <= 0x7f800000u) m = max(m, lo);
              if (hi <= 0x7f800000u) m = max(m, hi);
            }
            m = __reduce_max_sync(0xffffffffu, m);
            int ex = (int)(m >> 23) - 127;
            ex = kv::query_exponent(ex, m == 0);
            const float inv = a.scale < 0.f ? -kv::pow2f(-ex) : kv::pow2f(-ex);
            const int srow = 32 * (warp & 3) + r0 + r;
            unsigned char *dst = sQ + mt * Cfg::kQTile + srow * 128;
            // element d is at place p of its row: panel p / 64, swizzled 16-byte chunk
            auto at = [&](int p) {
              return dst + (p >> 6) * 16384 + (((p >> 3 & 7) ^ (srow & 7)) << 4) + (p & 7) * 2;
            };
            if constexpr (E == 2) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int d = lane * 2 + e;
                *reinterpret_cast<__half *>(at((d & ~3) + Widen<CODE>::place(d & 3))) =
                    __float2half_rn(f[e] * inv);
              }
            } else {
              uint32_t h[E / 2];
#pragma unroll
              for (int e = 0; e < E; e += 4) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[Widen<CODE>::place(j)] = f[e + j] * inv;
                h[e / 2] = half2_bits(y[0], y[1]);
                h[e / 2 + 1] = half2_bits(y[2], y[3]);
              }
              if constexpr (E == 8)
                *reinterpret_cast<uint4 *>(at(lane * 8)) = make_uint4(h[0], h[1], h[2], h[3]);
              else
                *reinterpret_cast<uint2 *>(at(lane * 4)) = make_uint2(h[0], h[1]);
            }
            if (r0 + r == lane) qa = fabsf(a.scale) * kLog2e * kv::pow2f(ex);
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_mma(&q_full);
      }
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t tO = tmem + lanes + Cfg::kO + mt * D;
      float M = -INFINITY, Ms = 0.f, L = 0.f;
      for (int j = 0; j < T && ok; ++j) {
        const uint32_t n = done + j, buf = MT == 2 ? mt : n & 1;
        const uint32_t tS = tmem + lanes + buf * kBN;
        const int info = n % kInfo;
        if (!warp_wait(&info_full[info], n / kInfo)) {
          ok = false;
          break;
        }
        const bool odd = s_odd[info] != 0;  // some V exponents far from the others
        if (!warp_wait(&s_full[buf], MT == 2 ? n : n >> 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const int open = lim - (w.begin + j) * kBN;  // columns that this row may see
        const bool masked = __any_sync(0xffffffffu, open < kBN);
        // One pass over S: weights under the present reference, their sum (in units of the
        // denominator) and the largest exponent, as far above the reference as it is.  `hide`:
        // some lane has columns that it may not see.
        uint32_t p[kBN / 2];
        float sum, peak;
        auto weigh = [&](auto hide) {
          uint32_t s[2][32];
          float top[2] = {-INFINITY, -INFINITY};
          sum = 0.f;
          tmem_ld32_async(tS, s[0]);
#pragma unroll
          for (int h = 0; h < kBN / 32; ++h) {
            tmem_ld_wait();
            if (h + 1 < kBN / 32) tmem_ld32_async(tS + 32 * (h + 1), s[(h + 1) & 1]);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t *v = s[h & 1] + 16 * b;
              const float f = qa * s_ks[info][2 * h + b], e = s_ve[info][2 * h + b] - Ms;
              float2 part = make_float2(0.f, 0.f);
#pragma unroll
              for (int x = 0; x < 16; x += 2) {
                float2 y =
                    fma2(make_float2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), f, e);
                if (hide.value) {
                  if (32 * h + 16 * b + x >= open) y.x = -INFINITY;
                  if (32 * h + 16 * b + x + 1 >= open) y.y = -INFINITY;
                }
                top[b] = fmaxf(fmaxf(y.x, y.y), top[b]);
                y.x = fast_exp2(y.x);
                y.y = fast_exp2(y.y);
                part = add2(part, y);
                p[16 * h + 8 * b + x / 2] = half2_bits(y.x, y.y);
              }
              sum = fmaf(part.x + part.y, s_un[info][2 * h + b], sum);
            }
          }
          peak = fmaxf(top[0], top[1]);
        };
        bool seen = MT == 2 || j == 0;  // pv_done of the tile before this one: with MT = 2 its
                                        // product came before this tile's S
        float apart = 0.f;
        bool todo = odd;
        for (int raises = 0;;) {  // again after the reference was raised (once, or twice if odd)
          if (masked)
            weigh(std::true_type{});
          else
            weigh(std::false_type{});
          const float limit = M == -INFINITY ? -INFINITY : kSlack + kLift;
          bool raise = __any_sync(0xffffffffu, peak > limit) && raises < (odd ? 2 : 1);
          if (!raise && !todo) break;
          if (odd) {
            const float2 x = weigh_apart(tS, open, qa, Ms, s_ks[info], s_ve[info]);
            apart = x.x;
            peak = fmaxf(peak, x.y);
            todo = raise = __any_sync(0xffffffffu, peak > limit) && raises < 2;
            if (!raise) continue;  // (for the weights, which are not kept over this)
          }
          ++raises;
          const float m = fmaxf(M, ceilf(peak + Ms));
          const float f = m == -INFINITY ? 1.f : fast_exp2(M - m);
          if (m != -INFINITY) L = kv::lower(L, M - m);
          M = m;
          Ms = m == -INFINITY ? 0.f : m - kLift;
          if (j > 0) {  // O holds the tiles before this one
            if (!seen && !warp_wait(&pv_done[mt], n - 1)) {
              ok = false;
              break;
            }
            seen = true;
            tc::fence_after_sync();
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              tmem_ld32_async(tO + x, o);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st16(tO + x, o);
              tmem_st16(tO + x + 16, o + 16);
            }
          }
        }
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < kBN / 2; x += 16) tmem_st16(tS + x, p + x);
        L += odd ? apart : sum;
        tc::tmem_st_wait();
        tc::fence_before_sync();
        if (!seen && !warp_wait(&pv_done[mt], n - 1)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) {
          arrive_mma(&p_full[mt]);
          mbar_arrive(&info_empty[info]);
        }
      }
      // ---- outputs ----
      if (ok && T > 0 && !warp_wait(&pv_done[mt], done + T - 1)) ok = false;
      const bool live = row < w.rows;
      const bool whole = splits == 1 || u >= hinted_units;
      float *mine = whole ? part : part + ((int64_t)block * splits + split) * Cfg::kPartFloats;
      if (!ok) {  // the join finds this and writes nothing
        if (!whole && live) mine[R * D + row] = kv::no_result();
      } else {
        tc::fence_after_sync();
        const int64_t at = (int64_t)(w.tok0 + grow / group) * a.ld_o +
                           (int64_t)(head * group + grow % group) * D;
        if (!whole) {
          if (live) {
            mine[R * D + row] = M;
            mine[R * D + R + row] = L;
          }
          mine += (int64_t)row * D;
        }
        const float inv = whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t o[32];
          float v[32];
          if (T > 0) {
            tmem_ld32_async(tO + x, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int y = 0; y < 32; ++y)
            v[y] = T > 0 ? __uint_as_float(o[(y & ~3) + Widen<CODE>::place(y & 3)]) * inv : 0.f;
          if (live) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              if (!whole)
                put8(mine + x + y, v + y);
              else if (a.o_dtype == GDN_F32)
                put8(static_cast<float *>(a.o) + at + x + y, v + y);
              else
                put8(static_cast<bf16 *>(a.o) + at + x + y, v + y);
            }
          }
        }
        tc::fence_before_sync();
      }
    });
  } else if (warp < kMma) {
    set_regs_down<Cfg::kConvRegs>();
    each_unit([&](const int64_t, const int T) {
      // ---- converters ----
      constexpr int kTeam = 32 * CW / TEAMS;
      constexpr int VPS = Cfg::kSlot / 32 / kTeam;  // loads (of 16 codes) per thread and slot
      const int team = (warp - kConv) / (CW / TEAMS);
      const int ct = tid - 32 * (kConv + team * (CW / TEAMS));
      // Place of a thread's load v in a slot of 4 or 8 columns of 16 codes: with 4, 4 lanes to
      // a row; with 8, lanes 0-3 and 8-11 share a row, 4-7 and 12-15 the next.  Either way
      // eight consecutive lanes write all eight 16-byte columns of the swizzled rows.
      auto place4 = [&](int v, int *row, int *col) {
        *row = v * (kTeam / 4) + (ct >> 2);
        *col = ct & 3;
      };
      auto place8 = [&](int v, int *row, int *col) {
        *row = v * (kTeam / 8) + ((ct >> 2 & 1) | (ct >> 3 & ~1));
        *col = (ct & 3) | (ct >> 1 & 4);
      };
      auto in_slot = [&](int side, int v, int *row, int *col) {
        if constexpr (!PAIR) {
          if constexpr (D == 64)
            place4(v, row, col);
          else
            place8(v, row, col);
        } else if (side == 0) {  // 64 tokens, d / 16 columns, by eights
          place8(D == 256 ? v % (VPS / 2) : v, row, col);
          if (D == 256 && v >= VPS / 2) *col += 8;
        } else if constexpr (D == 256) {
          place8(v, row, col);
        } else {
          place4(v, row, col);
        }
      };
      const int page_bytes = D << c.page_log2;
      const int n_slots = 2 * H * T;
      // slot x: its tile, side and half, in the order of the MMAs
      auto place = [&](int x, int *tile, int *side, int *half) {
        const int y = x / H;
        *half = x % H;
        if (MT == 2) {  // K0 V0 K1 V1 ...
          *tile = y >> 1;
          *side = y & 1;
        } else if (y == 0 || T == 1) {  // K0, K1 V0, K2 V1, ... V(T-1)
          *tile = 0;
          *side = y;
        } else if (y == 2 * T - 1) {
          *tile = T - 1;
          *side = 1;
        } else {
          *side = (y + 1) & 1;
          *tile = *side ? (y >> 1) - 1 : (y + 1) >> 1;
        }
      };
      uint4 code[VPS];
      auto load = [&](int x, uint4 *dst) {
        int tile, side, half;
        place(x, &tile, &side, &half);
        const uint32_t n = done + tile;
        const int info = n % kInfo;
        if (!warp_wait(&info_full[info], n / kInfo)) return false;
        // of a pair, this CTA takes half of K's tokens and half of V's d
        const int tok0 = PAIR && side == 0 ? rank * 64 : 0;
        const uint8_t *base =
            (side ? c.v : c.k) + (PAIR ? (side ? rank * (D / 2) : 0) : half * Cfg::DC);
        auto fetch = [&](int v, int r, int col, int blk) {
          const uint8_t *p =
              base + (int64_t)blk * page_bytes + (r & (c.page_tokens - 1)) * D + 16 * col;
          asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(dst[v].x), "=r"(dst[v].y), "=r"(dst[v].z), "=r"(dst[v].w)
                       : "l"(p));
        };
        const bool plain = s_plain[info] != 0;  // nothing of the tile to leave out
        int blk[VPS];
#pragma unroll
        for (int v = 0; v < VPS; ++v) {
          int r, col;
          in_slot(side, v, &r, &col);
          blk[v] = s_blk[info][(tok0 + r) >> 4];
        }
        // (the arrival comes before the loads: it would wait for them)
        __syncwarp();
        if (lane == 0) mbar_arrive(&info_empty[info]);
        if (plain) {  // loads without a branch between them
#pragma unroll
          for (int v = 0; v < VPS; ++v) {
            int r, col;
            in_slot(side, v, &r, &col);
            fetch(v, tok0 + r, col, blk[v]);
          }
        } else {
#pragma unroll
          for (int v = 0; v < VPS; ++v) {
            int r, col;
            in_slot(side, v, &r, &col);
            dst[v] = make_uint4(0, 0, 0, 0);  // past the end, or no page: the code of zero
            if (blk[v] >= 0 && (w.begin + tile) * kBN + tok0 + r < w.kv_len)
              fetch(v, tok0 + r, col, blk[v]);
          }
        }
        return true;
      };
      if (team < n_slots) ok = load(team, code);
      for (int x = team; x < n_slots && ok; x += TEAMS) {
        const uint32_t n = slots + x;
        if (n >= NS && !warp_wait(&slot_empty[n % NS], n / NS - 1)) {
          ok = false;
          break;
        }
        int tile, side, half;
        place(x, &tile, &side, &half);
        const int panel = side ? 16384 : Cfg::kKPanel;
        unsigned char *dst = sKV + (n % NS) * Cfg::kSlot;
#pragma unroll
        for (int v = 0; v < VPS; ++v) {
          int r, col;
          in_slot(side, v, &r, &col);
          uint32_t h[8];
          Widen<CODE>::four(code[v].x, h[0], h[1]);
          Widen<CODE>::four(code[v].y, h[2], h[3]);
          Widen<CODE>::four(code[v].z, h[4], h[5]);
          Widen<CODE>::four(code[v].w, h[6], h[7]);
          unsigned char *q = dst + (col >> 2) * panel + r * 128;
          const int k = 2 * (col & 3);
          *reinterpret_cast<uint4 *>(q + ((k ^ (r & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(q + (((k + 1) ^ (r & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_mma(&slot_full[n % NS]);
        if (x + TEAMS < n_slots) ok = load(x + TEAMS, code);
      }
    });
  } else if (warp == kMma) {
    set_regs_down<Cfg::kMiscRegs>();
    each_unit([&](const int64_t, const int T) {
      // ---- MMA ----
      // The whole warp takes every branch and wait; one elected lane issues.  (Issued
      // from a branch on the lane number, an MMA took 160 cycles under busy softmax
      // warps instead of 70.)
      if (T > 0 && rank == 0) {
        constexpr int kM = 128 * Cfg::kCtas;
        constexpr uint32_t id_qk = idesc_f16(kM, kBN, false);
        constexpr uint32_t id_pv = idesc_f16(kM, PAIR ? D : Cfg::DC, true);
        const bool issue = elect_one();
        uint32_t at = slots;  // next slot
        auto next_slot = [&]() {
          const bool got = warp_wait(&slot_full[at % NS], at / NS);
          tc::fence_after_sync();
          return got;
        };
        const uint32_t q_low = desc_low(smem_addr(sQ), 16);
        const uint32_t k_low = desc_low(smem_addr(sKV), 16);
        const uint32_t v_low = desc_low(smem_addr(sKV), 16384);
        // S (+)= Q K^T of one slot; `then`: what to commit to
        auto qk = [&](uint32_t slot, int half, int mt, int buf, uint64_t *then, uint64_t *free) {
          const uint32_t q = q_low + (mt * Cfg::kQTile + half * (Cfg::DC / 64) * 16384) / 16;
          const uint32_t k = k_low + (slot % NS) * (Cfg::kSlot / 16);
          if (issue) {
#pragma unroll
            for (int x = 0; x < D / H / 16; ++x)
              mma_ss<PAIR>(tmem + buf * kBN, desc(q + ((x >> 2) * 16384 + (x & 3) * 32) / 16),
                           desc(k + ((x >> 2) * Cfg::kKPanel + (x & 3) * 32) / 16), id_qk,
                           half + x > 0);
            if (then) mma_commit<PAIR>(then);
            if (free) mma_commit<PAIR>(free);
          }
          __syncwarp();
        };
        // O (+)= P V of one slot
        auto pv = [&](uint32_t slot, int half, int mt, int buf, bool first, uint64_t *then,
                      uint64_t *free) {
          const uint32_t v = v_low + (slot % NS) * (Cfg::kSlot / 16);
          if (issue) {
#pragma unroll
            for (int x = 0; x < kBN / 16; ++x)
              mma_ts<PAIR>(tmem + Cfg::kO + mt * D + half * Cfg::DC, tmem + buf * kBN + 8 * x,
                           desc(v + x * 128), id_pv, !first || x > 0);
            if (then) mma_commit<PAIR>(then);
            if (free) mma_commit<PAIR>(free);
          }
          __syncwarp();
        };
        auto p_ready = [&](int mt, int j) {
          const bool got = warp_wait(&p_full[mt], done + j);
          tc::fence_after_sync();
          return got;
        };
        auto run = [&]() {
          if (!warp_wait(&q_full, units)) return false;
          tc::fence_after_sync();
          if constexpr (MT == 2) {
            if (!next_slot()) return false;
            qk(at, 0, 0, 0, &s_full[0], nullptr);
            qk(at, 0, 1, 1, &s_full[1], &slot_empty[at % NS]);
            ++at;
            for (int j = 0; j < T; ++j) {  // `at`: V of tile j, then K of the next
              if (!next_slot() || !p_ready(0, j)) return false;
              pv(at, 0, 0, 0, j == 0, &pv_done[0], nullptr);
              if (j + 1 < T) {
                ++at;
                if (!next_slot()) return false;
                qk(at, 0, 0, 0, &s_full[0], nullptr);
                --at;
              }
              if (!p_ready(1, j)) return false;
              pv(at, 0, 1, 1, j == 0, &pv_done[1], &slot_empty[at % NS]);
              ++at;
              if (j + 1 < T) {
                qk(at, 0, 1, 1, &s_full[1], &slot_empty[at % NS]);
                ++at;
              }
            }
          } else {
            for (int j = -1; j < T; ++j) {
              if (j + 1 < T) {
                const uint32_t n = done + j + 1;
                for (int h = 0; h < H; ++h, ++at) {
                  if (!next_slot()) return false;
                  qk(at, h, 0, n & 1, h == H - 1 ? &s_full[n & 1] : nullptr, &slot_empty[at % NS]);
                }
              }
              if (j >= 0) {
                if (!p_ready(0, j)) return false;
                for (int h = 0; h < H; ++h, ++at) {
                  if (!next_slot()) return false;
                  pv(at, h, 0, (done + j) & 1, j == 0, h == H - 1 ? &pv_done[0] : nullptr,
                     &slot_empty[at % NS]);
                }
              }
            }
          }
          return true;
        };
        ok = run();
        if (!ok) {  // the MMAs in flight finish before TMEM is freed
          if (issue) mma_commit<PAIR>(&drain);
          mbar_wait_bounded(&drain, 0);
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    });
  } else if (warp == kPages) {
    set_regs_down<Cfg::kMiscRegs>();
    each_unit([&](const int64_t, const int T) {
      // ---- page ids and scales, four tiles at a time ----
      const int32_t *table = c.table + (int64_t)w.slot * c.max_pages;
      int e_max = kv::kLowExp;  // largest V exponent of the unit's tiles so far
      for (int j0 = 0; j0 < T && ok; j0 += 4) {
        const int j = j0 + (lane >> 3), gr = lane & 7;
        const int tok = (w.begin + j) * kBN + 16 * gr;
        int blk = -1;
        float ks = 0.f, ve = -INFINITY, un = 0.f;
        int e = e_max;
        if (j < T && tok < w.kv_len) {
          const int id = table[tok >> c.page_log2];
          if (id >= 0 && id < c.n_pages) {
            blk = (int)c.block(layer, id, head);
            ks = c.k_scale[blk];
            e = kv::scale_exponent<CODE>(c.v_scale[blk]);
            ve = (float)e;
            un = kv::pow2f(-e);
          } else {
            raise_error(c.err, GDN_DEVERR_PAGE);
          }
        }
        e_max = __reduce_max_sync(0xffffffffu, max(e, e_max));
        const bool odd_group = blk >= 0 && e < max(kv::kLowExp, e_max - kv::kFar);
        for (int x = 0; x < 4 && j0 + x < T && ok; ++x) {
          const uint32_t n = done + j0 + x;
          const int info = n % kInfo;
          if (n >= kInfo) ok = warp_wait(&info_empty[info], n / kInfo - 1);
          if (!ok) break;
          const bool plain =
              __all_sync(0xffffffffu, (lane >> 3) != x || (blk >= 0 && tok + 16 <= w.kv_len));
          const bool odd = __any_sync(0xffffffffu, (lane >> 3) == x && odd_group);
          if ((lane >> 3) == x) {
            s_plain[info] = plain;
            s_odd[info] = odd;
            s_blk[info][gr] = blk;
            s_ks[info][gr] = ks;
            s_ve[info][gr] = ve;
            s_un[info][gr] = un;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&info_full[info]);
        }
      }
    });
  } else {
    set_regs_down<Cfg::kMiscRegs>();
  }
  __syncwarp();
  tc::fence_before_sync();
  if constexpr (PAIR)
    cluster_sync();  // no CTA leaves while the other's arrivals or MMAs may still reach it
  else
    __syncthreads();
  if (warp == kMma) {
    tc::fence_after_sync();
    tmem_dealloc<PAIR>(tmem, Cfg::kTmem);
  }
}

// The units by weight, the heaviest first, so that the last CTAs to end have little to do
// (for several sequences in more than one wave: a sequence's units weigh what its context
// does).  One CTA: a histogram over the tile counts, and a scatter; units of equal weight
// come in any order, which no result depends on.
constexpr int kOrderThreads = 1024;
constexpr int kOrderMost = 65536;  // units

template <int R>
__global__ void __launch_bounds__(kOrderThreads)
    order_units_kernel(const KVView c, const KVAttendArgs a, const int units, const int shift,
                       int *order) {
  __shared__ int bins[kOrderThreads], sums[32];
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.seq.n_seqs * c.h_kv, total = units * heads;
  // place `v`: row tile v / heads of sequence and head v % heads; bin 0 is the heaviest
  auto bin = [&](int v) {
    Unit w;
    const int z = v % heads;
    if (!find_unit(c, a, z / c.h_kv, z % c.h_kv, v / heads, R, 0, 1, false, &w))
      return kOrderThreads - 1;
    return max(kOrderThreads - 2 - (w.tiles >> shift), 0);
  };
  bins[tid] = 0;
  __syncthreads();
  for (int v = tid; v < total; v += kOrderThreads) atomicAdd(&bins[bin(v)], 1);
  __syncthreads();
  const int own = bins[tid];
  int x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  for (int k = 0; k < warp; ++k) x += sums[k];
  bins[tid] = x - own;  // where the bin begins
  __syncthreads();
  for (int v = tid; v < total; v += kOrderThreads) order[atomicAdd(&bins[bin(v)], 1)] = v;
}

// Joins the splits of a unit: a CTA per (unit, sequence and head) and four rows.
constexpr int kJoinRows = 4;

template <int D, int R>
__global__ void __launch_bounds__(kJoinRows * D / 4)
    attend_prompt_join_kernel(const KVView c, const KVAttendArgs a, const int splits,
                              const float *part) {
  constexpr int kPartFloats = R * (D + 2);
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int heads = a.seq.n_seqs * c.h_kv, z = blockIdx.x % heads;
  Unit w;
  if (!find_unit(c, a, z / c.h_kv, z % c.h_kv, blockIdx.x / heads, R, 0, 1, false, &w)) return;
  const int row = blockIdx.y * kJoinRows + threadIdx.x / (D / 4);
  const int d = 4 * (threadIdx.x % (D / 4));
  if (row >= w.rows) return;
  const float *base = part + (int64_t)blockIdx.x * splits * kPartFloats;
  float m = -INFINITY, l = 0.f;
  bool missing = false;
  for (int s = 0; s < splits; ++s) {
    const float pm = __ldcg(base + (int64_t)s * kPartFloats + R * D + row);
    missing |= pm != pm;
    m = fmaxf(m, pm);
  }
  if (missing) return;  // some part gave up: the row stays as it was
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float *p = base + (int64_t)s * kPartFloats;
    const float pm = __ldcg(p + R * D + row), pl = __ldcg(p + R * D + R + row);
    const float f = kv::join_factor(pl, pm, m);
    l += kv::join_sum(pl, pm, m);
    sum = axpby4(1.f, sum, f, __ldcg(reinterpret_cast<const float4 *>(p + (int64_t)row * D + d)));
  }
  const int group = c.h_q / c.h_kv, grow = w.row0 + row;
  const int64_t at = (int64_t)(w.tok0 + grow / group) * a.ld_o +
                     (int64_t)(w.head * group + grow % group) * D + d;
  const float4 v = scale4(l == 0.f ? 0.f : 1.f / l, sum);
  if (a.o_dtype == GDN_F32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at) = v;
  } else {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<bf16 *>(a.o) + at) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
  }
}

template <int CODE, int D, int MT, bool PAIR>
cudaError_t launch_prompt(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                          cudaStream_t s) {
  using Cfg = PromptCfg<D, MT, PAIR>;
  auto kernel = attend_prompt_kernel<CODE, D, MT, PAIR>;
  static std::atomic<uint64_t> seen{0};
  cudaError_t e = kv::allow_smem(kernel, Cfg::kSmem, h.device, seen);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.max_seqlen * (c.h_q / c.h_kv);
  const int64_t z = (int64_t)a.seq.n_seqs * c.h_kv;
  int64_t units = (rows + Cfg::kRows - 1) / Cfg::kRows;
  if (units * z > INT32_MAX / Cfg::kCtas) units = INT32_MAX / Cfg::kCtas / z;
  // too few units for the GPU: cut each one's context
  const int64_t tiles = a.max_kv_len / kBN + 1, room = h.sm_count / Cfg::kCtas;
  int64_t splits = 1;
  if (units * z < room) {
    splits = room / (units * z);
    if (splits > tiles / 3) splits = tiles / 3;
    if (splits > 64) splits = 64;
    if (splits < 1) splits = 1;
  }
  const bool sort = a.seq.n_seqs > 1 && units * z > room && units * z <= kOrderMost;
  void *work = nullptr;
  bool temporary = false;
  if (splits > 1 || sort) {
    const size_t bytes = sort ? (size_t)units * z * sizeof(int)
                              : (size_t)z * units * splits * Cfg::kPartFloats * sizeof(float);
    e = h.work->get(bytes, s, &work, &temporary);
    if (e != cudaSuccess) return e;
  }
  if (sort) {
    int shift = 0;
    while ((tiles >> shift) > kOrderThreads - 2) ++shift;
    e = kv::launch(order_units_kernel<Cfg::kRows>, dim3(1), kOrderThreads, 0, s, 1, c, a,
                   (int)units, shift, static_cast<int *>(work));
    if (e != cudaSuccess) {
      if (temporary) cudaFreeAsync(work, s);
      return e;
    }
  }
  e = kv::launch(kernel, dim3((unsigned)(units * z * Cfg::kCtas), (unsigned)splits), Cfg::kThreads,
                 Cfg::kSmem, s, Cfg::kCtas, c, layer, a, (int)splits, (int)units,
                 sort ? static_cast<const int *>(work) : nullptr, static_cast<float *>(work));
  if (splits > 1 && e == cudaSuccess)
    e = kv::launch(attend_prompt_join_kernel<D, Cfg::kRows>,
                   dim3((unsigned)(units * z), Cfg::kRows / kJoinRows), kJoinRows * D / 4, 0, s, 1,
                   c, a, (int)splits, static_cast<const float *>(work));
  const cudaError_t ef = temporary ? cudaFreeAsync(work, s) : cudaSuccess;
  return e != cudaSuccess ? e : ef;
}

template <int CODE>
cudaError_t by_dim(const KVView &c, int layer, const KVAttendArgs &a, const KVHost &h,
                   cudaStream_t s) {
  const int64_t rows = (int64_t)a.max_seqlen * (c.h_q / c.h_kv);
  if (c.d == 256)
    return rows <= 128 ? launch_prompt<CODE, 256, 1, false>(c, layer, a, h, s)
                       : launch_prompt<CODE, 256, 1, true>(c, layer, a, h, s);
  if (c.d == 128)
    return rows <= 128   ? launch_prompt<CODE, 128, 1, false>(c, layer, a, h, s)
           : rows <= 256 ? launch_prompt<CODE, 128, 2, false>(c, layer, a, h, s)
                         : launch_prompt<CODE, 128, 2, true>(c, layer, a, h, s);
  return rows <= 128 ? launch_prompt<CODE, 64, 1, false>(c, layer, a, h, s)
                     : launch_prompt<CODE, 64, 2, false>(c, layer, a, h, s);
}

}  // namespace

cudaError_t launch_kv_attend_prompt(const KVView &c, int layer, const KVAttendArgs &a,
                                    const KVHost &h, cudaStream_t s) {
  return c.code == GDN_KV_I8 ? by_dim<GDN_KV_I8>(c, layer, a, h, s)
                             : by_dim<GDN_KV_E4M3>(c, layer, a, h, s);
}

}  // namespace gdn
