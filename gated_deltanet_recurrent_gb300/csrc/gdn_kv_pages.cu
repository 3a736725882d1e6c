// Pages of the KV cache handed out and taken back on the GPU.
//
// Grow.  Sequence i needs need_i = max(0, ceil((pos_i + len_i) / P) - held_i) pages and is granted
// them iff need_i = 0 or need_0 + ... + need_i <= n_free: the sequences are served in order, and
// one that cannot be served stops all after it that need any.  So the granted pages, counted
// through the call, are k = need_0 + ... + need_(i-1), ... , and page k is free[n_free - 1 - k].
// Trim gives back the pages beyond ceil(len_i / P); page k of K goes to free[n_free + K - 1 - k], so
// that a grow of the same sequences finds the same pages again.
//
// There is next to nothing to move (8 bytes a page, 12 a token that is mapped): what counts is the
// chain slot -> held -> scan -> free page.  So every CTA reads all sequences and scans them itself,
// 1024 at a time and a thread each, and then fills its share of the table and of the tokens' rows,
// found by binary search in the scan.  No CTA waits for another: what the scans read (held, n_free)
// is written by the CTA that ends last, which it learns from a ticket.  A call of few tokens is one
// CTA, without a ticket.  Measured, trim and grow together, call by call: one sequence 9.4 us (8.0 of them
// on the GPU), a decode step of 256 9.6, 64 prompts of up to 8192 tokens (310 000 tokens, 20 000 pages of
// 16) 17.2.
#include <new>
#include <vector>

#include "gdn_handles.h"
#include "gdn_host.h"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 1024;

struct Book {
  int32_t *table, *held, *free_pages, *n_free;
};

// The sequences of one round of the scan.
struct Round {
  int first[kThreads];     // pages of the call before this sequence's
  int have[kThreads];      // grow: pages it holds; trim: pages it keeps
  int slot[kThreads];
  int pos[kThreads];       // -1: the entry is skipped
  int tok[kThreads + 1];   // its first token; the next one's, which it ends before
  unsigned char granted[kThreads];
};

// Slots of the call, and those that it names more than once.
struct Slots {
  uint32_t seen[2048], twice[2048];
};

// Inclusive sum over the CTA's threads; *total: of all.  s: a place per warp.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t *s, int64_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s[warp] = x;
  __syncthreads();
  int64_t w = s[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // s may be written again
  return x + (warp > 0 ? before : 0);
}

// The last of a[0..n) that is <= k (a[0] <= k).
__device__ __forceinline__ int last_at_most(const int *a, int n, int k) {
  int lo = 0;
  while (n > 1) {
    const int half = n >> 1;
    if (a[lo + half] <= k) lo += half;
    n -= half;
  }
  return lo;
}

// Marks the call's slots, of which this thread has `own` already.  A slot that it names twice is none
// of its entries' (they would hand out or give back the same pages twice).
__device__ __forceinline__ void mark_slots(const KVView &c, const int32_t *slot_ids, int n, int own,
                                           Slots &m) {
  for (int w = threadIdx.x; w <= (c.n_slots - 1) >> 5; w += kThreads) m.seen[w] = m.twice[w] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int slot = i < kThreads ? own : slot_ids[i];
    if (slot < 0 || slot >= c.n_slots) continue;
    const uint32_t bit = 1u << (slot & 31);
    if (atomicOr(&m.seen[slot >> 5], bit) & bit) atomicOr(&m.twice[slot >> 5], bit);
  }
  __syncthreads();
}

__device__ __forceinline__ bool slot_ok(const KVView &c, const Slots &m, int slot, bool report) {
  const bool good = slot >= 0 && slot < c.n_slots && !(m.twice[slot >> 5] >> (slot & 31) & 1);
  if (!good && report) raise_error(c.err, GDN_DEVERR_SLOT);
  return good;
}

// The number of free pages, or 0 where the book's count cannot be one.
__device__ __forceinline__ int free_count(const KVView &c, const Book &b, bool *bad) {
  const int top = *b.n_free;
  *bad = top < 0 || top > c.n_pages;
  if (*bad && blockIdx.x + threadIdx.x == 0) raise_error(c.err, GDN_DEVERR_PAGE);
  return *bad ? 0 : top;
}

// True in the CTA that passes here last; what the others read before, it may now write.
__device__ __forceinline__ bool last_here(unsigned int *ticket, int *flag) {
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    *flag = atomicAdd(ticket, 1u) == gridDim.x - 1;
    if (*flag) *ticket = 0;
    __threadfence();
  }
  __syncthreads();
  return *flag != 0;
}

__global__ void __launch_bounds__(kThreads)
    grow_kernel(KVView c, Book b, SeqIndex seq, const int32_t *__restrict__ pos,
                int32_t *__restrict__ positions, int64_t *__restrict__ rows,
                int32_t *__restrict__ granted) {
  __shared__ Slots marks;
  __shared__ Round r;
  __shared__ int64_t s_scan[32];
  __shared__ int s_last, s_taken;
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int tid = threadIdx.x, n = seq.n_seqs;
  const bool lead = blockIdx.x == 0;
  // a sequence as it is in memory; what it takes is on its way before anything is looked at
  int slot = -1, first = -1, t0 = 0, t1 = 0, have = 0;
  auto fetch = [&](int i) {
    if (i >= n) return;
    slot = seq.slot_ids[i];
    first = pos[i];
    t0 = seq.cu_seqlens ? seq.cu_seqlens[i] : i;
    t1 = seq.cu_seqlens ? seq.cu_seqlens[i + 1] : i + 1;
    have = slot >= 0 && slot < c.n_slots ? b.held[slot] : 0;
  };
  fetch(tid);
  bool bad_count;
  const int top = free_count(c, b, &bad_count);
  mark_slots(c, seq.slot_ids, n, slot, marks);

  // Sequences [base, base + 1024): their entries of `r`, and the pages asked for so far.  Returns
  // the pages granted to this thread's.
  auto read_round = [&](int base, int64_t *asked, bool fetched, bool report) {
    const int i = base + tid;
    int need = 0;
    if (!fetched) fetch(i);
    if (i < n) {
      if (!slot_ok(c, marks, slot, report)) {
        first = -1;
      } else if (t0 < 0 || t1 < t0 || t1 > seq.total_tokens || first < 0 ||
                 (int64_t)first + (t1 - t0) > c.capacity()) {
        if (report) raise_error(c.err, GDN_DEVERR_SEQ);
        first = -1;
      } else {
        if (have < 0 || have > c.max_pages) {
          if (report) raise_error(c.err, GDN_DEVERR_PAGE);
          first = -1;
        } else {
          need = max(0, ((first + (t1 - t0) + c.page_tokens - 1) >> c.page_log2) - have);
          if (t1 == t0) need = 0;
        }
      }
    }
    int64_t total;
    const int64_t upto = *asked + scan(need, s_scan, &total);
    const bool got = i < n && first >= 0 && (need == 0 || upto <= top);
    r.first[tid] = (int)min(upto - need, (int64_t)INT32_MAX);
    r.have[tid] = have;
    r.slot[tid] = slot;
    r.pos[tid] = first;
    if (i < n) {
      r.tok[tid] = t0;
      if (tid + 1 == kThreads || i + 1 == n) r.tok[tid + 1] = t1;
    }
    r.granted[tid] = got;
    if (tid == 0) s_taken = 0;
    __syncthreads();
    if (got && need > 0) atomicMax(&s_taken, (int)upto);
    *asked += total;
    __syncthreads();
    return got ? need : 0;
  };

  const int step = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
  int64_t asked = 0;
  int taken = 0, need = 0;
  for (int base = 0; base < n; base += kThreads) {
    const int cnt = min(kThreads, n - base);
    need = read_round(base, &asked, base == 0, lead);
    if (lead && granted != nullptr && tid < cnt) granted[base + tid] = r.granted[tid];
    // the table entries of this round's pages
    for (int k = taken + me; k < s_taken; k += step) {
      const int j = last_at_most(r.first, cnt, k);
      const int id = b.free_pages[top - 1 - k];
      if (id < 0 || id >= c.n_pages) raise_error(c.err, GDN_DEVERR_PAGE);
      b.table[(int64_t)r.slot[j] * c.max_pages + r.have[j] + (k - r.first[j])] = id;
    }
    // the tokens, each once: those of no sequence are left as they are
    if (positions != nullptr || rows != nullptr) {
      const int hi = min(r.tok[cnt], seq.total_tokens);
      for (int64_t t64 = (int64_t)max(r.tok[0], 0) + me; t64 < hi; t64 += step) {
        const int t = (int)t64, j = last_at_most(r.tok, cnt, t);
        // (a malformed range has no tokens, and offsets that decrease may lead here from anywhere)
        if (r.tok[j] < 0 || t < r.tok[j] || t >= r.tok[j + 1] || r.tok[j + 1] > seq.total_tokens)
          continue;
        int p = -1;
        int64_t row = -1;
        if (r.pos[j] >= 0) {
          p = r.pos[j] + (t - r.tok[j]);
          if (r.granted[j]) {
            const int col = p >> c.page_log2, more = col - r.have[j];
            const int id = more < 0 ? b.table[(int64_t)r.slot[j] * c.max_pages + col]
                                    : b.free_pages[top - 1 - (r.first[j] + more)];
            if (id >= 0 && id < c.n_pages)
              row = ((int64_t)id << c.page_log2) + (p & (c.page_tokens - 1));
            else
              raise_error(c.err, GDN_DEVERR_PAGE);
          }
        }
        if (positions != nullptr) positions[t] = p;
        if (rows != nullptr) rows[t] = row;
      }
    }
    taken = max(taken, s_taken);
    if (gridDim.x == 1 && need > 0) b.held[r.slot[tid]] = r.have[tid] + need;
    __syncthreads();
  }
  if (!last_here(c.err + 1, &s_last)) return;
  if (gridDim.x > 1 && n <= kThreads) {  // the only round is the one in `r`
    if (need > 0) b.held[r.slot[tid]] = r.have[tid] + need;
  } else if (gridDim.x > 1) {
    asked = 0;
    for (int base = 0; base < n; base += kThreads) {
      need = read_round(base, &asked, false, false);
      if (need > 0) b.held[r.slot[tid]] = r.have[tid] + need;
      __syncthreads();
    }
  }
  if (tid == 0 && taken > 0) *b.n_free = top - taken;
}

__global__ void __launch_bounds__(kThreads)
    trim_kernel(KVView c, Book b, const int32_t *__restrict__ slot_ids,
                const int32_t *__restrict__ lens, int n) {
  __shared__ Slots marks;
  __shared__ Round r;
  __shared__ int64_t s_scan[32];
  __shared__ int s_last;
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  int slot = -1, len = 0, have = 0;  // as in grow_kernel
  auto fetch = [&](int i) {
    if (i >= n) return;
    slot = slot_ids[i];
    len = lens[i];
    have = slot >= 0 && slot < c.n_slots ? b.held[slot] : 0;
  };
  fetch(tid);
  bool bad_count;
  const int top = free_count(c, b, &bad_count);
  mark_slots(c, slot_ids, n, slot, marks);

  // Sequences [base, base + 1024): their entries of `r`, and the pages dropped so far.  Returns
  // the pages that this thread's drops.
  auto read_round = [&](int base, int64_t *dropped, bool report) {
    const int i = base + tid;
    int drop = 0, keep = 0;
    if (n > kThreads) fetch(i);
    if (i < n) {
      if (!slot_ok(c, marks, slot, report)) {
      } else if (len < 0) {
        if (report) raise_error(c.err, GDN_DEVERR_SEQ);
      } else {
        keep = (int)(((int64_t)len + c.page_tokens - 1) >> c.page_log2);
        if (have >= 0 && have <= c.max_pages)
          drop = max(0, have - keep);
        else if (report)
          raise_error(c.err, GDN_DEVERR_PAGE);
      }
    }
    int64_t total;
    const int64_t upto = *dropped + scan(drop, s_scan, &total);
    r.first[tid] = (int)min(upto - drop, (int64_t)INT32_MAX);
    r.have[tid] = keep;
    r.slot[tid] = slot;
    *dropped += total;
    __syncthreads();
    return drop;
  };

  int64_t all = 0;
  int drop = 0;
  for (int base = 0; base < n; base += kThreads) drop = read_round(base, &all, lead);
  // more pages than there are: the counts are not what they should be, and nothing is moved
  const bool sound = !bad_count && top + all <= c.n_pages;
  if (!sound && lead && tid == 0) raise_error(c.err, GDN_DEVERR_PAGE);
  const int step = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
  int64_t upto = 0;
  for (int base = 0; sound && base < n; base += kThreads) {
    const int64_t before = upto;
    if (n > kThreads)
      drop = read_round(base, &upto, false);
    else
      upto = all;  // its round is the one in `r`
    const int cnt = min(kThreads, n - base);
    for (int64_t k = before + me; k < upto; k += step) {
      const int j = last_at_most(r.first, cnt, (int)k);
      int32_t *entry = b.table + (int64_t)r.slot[j] * c.max_pages + r.have[j] + ((int)k - r.first[j]);
      const int id = *entry;
      if (id < 0 || id >= c.n_pages) raise_error(c.err, GDN_DEVERR_PAGE);
      b.free_pages[top + all - 1 - k] = id;
      *entry = -1;
    }
    if (gridDim.x == 1 && drop > 0) b.held[r.slot[tid]] = r.have[tid];
    __syncthreads();
  }
  if (!last_here(c.err + 1, &s_last) || !sound) return;
  if (gridDim.x > 1 && n <= kThreads) {
    if (drop > 0) b.held[r.slot[tid]] = r.have[tid];
  } else if (gridDim.x > 1) {
    upto = 0;
    for (int base = 0; base < n; base += kThreads) {
      drop = read_round(base, &upto, false);
      if (drop > 0) b.held[r.slot[tid]] = r.have[tid];
      __syncthreads();
    }
  }
  if (tid == 0 && all > 0) *b.n_free = top + (int)all;
}

// CTAs for `items` table entries or tokens, `each` a thread, and no more CTAs than run at once.
int grid_for(int64_t items, int each, int sm_count) {
  const int64_t ctas = (items + each * kThreads - 1) / (each * kThreads);
  return (int)(ctas < 1 ? 1 : ctas > sm_count ? sm_count : ctas);
}

}  // namespace
}  // namespace gdn

namespace {

using namespace gdn::host;

gdn_status check_book(const gdn_kv *c, const gdn_kv_pages *b) {
  if (!c) return fail(GDN_ERR_ARG, "kv is NULL");
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != c->device)
    return fail(GDN_ERR_ARG, "current device %d is not the cache's device %d", dev, c->device);
  if (!b || !b->page_table || !b->held || !b->free_pages || !b->n_free)
    return fail(GDN_ERR_ARG, "pages and its four arrays must be non-NULL");
  if (b->page_table != c->view.table)
    return fail(GDN_ERR_ARG, "pages->page_table is not the cache's page table");
  if (((uintptr_t)b->held | (uintptr_t)b->free_pages | (uintptr_t)b->n_free) % 4)
    return fail(GDN_ERR_ARG, "held, free_pages and n_free must be 4-byte aligned");
  gdn_status st;
  if (c->desc.host_checks && ((st = check_device_ptr(b->held, "held")) ||
                              (st = check_device_ptr(b->free_pages, "free_pages")) ||
                              (st = check_device_ptr(b->n_free, "n_free"))))
    return st;
  return GDN_OK;
}

// Host checks: slots in range and distinct, the book's counts possible, the
// lengths (cu: of positions starts[i], ... within a slot) in range, and so the
// pages that change hands.
gdn_status check_arrays(const gdn_kv *c, const gdn_kv_pages *b, const int32_t *slot_ids,
                        const int32_t *starts, const char *name, bool growing,
                        const int32_t *cu_seqlens, int n, int total, cudaStream_t s) {
  const gdn_kv_desc &d = c->desc;
  std::vector<int32_t> slots, from, cu, held, count, pages;
  gdn_status st;
  if ((st = fetch(slots, slot_ids, (size_t)n, s, "slot_ids")) ||
      (st = fetch(from, starts, (size_t)n, s, name)) ||
      (st = fetch(held, b->held, (size_t)d.n_slots, s, "held")) ||
      (st = fetch(count, b->n_free, 1, s, "n_free")) ||
      (st = growing ? fetch(pages, b->free_pages, (size_t)d.n_pages, s, "free_pages")
                    : fetch(pages, b->page_table, (size_t)d.n_slots * d.max_pages, s, "page_table")))
    return st;
  const auto valid = [&](int32_t id) { return id >= 0 && id < d.n_pages; };
  if (count[0] < 0 || count[0] > d.n_pages)
    return fail(GDN_ERR_SIZE, "n_free = %d outside [0, %d]", count[0], d.n_pages);
  if (cu_seqlens) {
    if ((st = fetch(cu, cu_seqlens, (size_t)n + 1, s, "cu_seqlens"))) return st;
    if (cu[0] != 0) return fail(GDN_ERR_SIZE, "cu_seqlens[0] = %d, expected 0", cu[0]);
    for (int i = 0; i < n; ++i)
      if (cu[i + 1] < cu[i]) return fail(GDN_ERR_SIZE, "cu_seqlens decreases at %d", i);
    if (cu[n] != total)
      return fail(GDN_ERR_SIZE, "cu_seqlens[%d] = %d, expected total_tokens %d", n, cu[n], total);
  }
  std::vector<unsigned char> seen((size_t)d.n_slots, 0);
  int64_t back = count[0], asked = 0, given = 0;
  for (int i = 0; i < n; ++i) {
    const int slot = slots[i];
    if (slot < 0 || slot >= d.n_slots)
      return fail(GDN_ERR_SLOT, "slot_ids[%d] = %d outside [0, %d)", i, slot, d.n_slots);
    if (seen[slot]) return fail(GDN_ERR_DUP_SLOT, "slot id %d repeated (entry %d)", slot, i);
    seen[slot] = 1;
    if (held[slot] < 0 || held[slot] > d.max_pages)
      return fail(GDN_ERR_SIZE, "held[%d] = %d outside [0, %d]", slot, held[slot], d.max_pages);
    const int64_t len = !growing ? 0 : cu_seqlens ? cu[i + 1] - cu[i] : 1;
    if (from[i] < 0 || (growing && from[i] + len > c->view.capacity()))
      return fail(GDN_ERR_SIZE, "%s[%d] = %d: outside the slot's %lld positions", name, i, from[i],
                  (long long)c->view.capacity());
    const int64_t keep = ((int64_t)from[i] + len + d.page_tokens - 1) / d.page_tokens;
    if (growing && len > 0 && keep > held[slot]) {
      asked += keep - held[slot];
      for (; asked <= count[0] && given < asked; ++given)
        if (!valid(pages[count[0] - 1 - given]))
          return fail(GDN_ERR_SIZE, "free_pages[%lld] = %d outside [0, %d)",
                      (long long)(count[0] - 1 - given), pages[count[0] - 1 - given], d.n_pages);
    }
    for (int64_t col = keep; !growing && col < held[slot]; ++col, ++back)
      if (!valid(pages[(size_t)slot * d.max_pages + col]))
        return fail(GDN_ERR_SIZE, "page_table[%d][%lld] = %d outside [0, %d)", slot, (long long)col,
                    pages[(size_t)slot * d.max_pages + col], d.n_pages);
  }
  if (back > d.n_pages)
    return fail(GDN_ERR_SIZE, "%lld pages would be free of %d", (long long)back, d.n_pages);
  return GDN_OK;
}

// No exception leaves a C entry point.
gdn_status check_host(const gdn_kv *c, const gdn_kv_pages *b, const int32_t *slot_ids,
                      const int32_t *starts, const char *name, bool growing,
                      const int32_t *cu_seqlens, int n, int total, cudaStream_t s) {
  try {
    return check_arrays(c, b, slot_ids, starts, name, growing, cu_seqlens, n, total, s);
  } catch (const std::bad_alloc &) {
    return fail(GDN_ERR_SIZE, "no host memory to check the index arrays");
  }
}

}  // namespace

extern "C" {

gdn_status gdn_kv_pages_grow(gdn_kv *c, const gdn_kv_pages *b, const int32_t *slot_ids,
                             const int32_t *pos, const int32_t *cu_seqlens, int32_t n_seqs,
                             int32_t total_tokens, int32_t *positions, int64_t *rows,
                             int32_t *granted, gdn_stream stream) {
  gdn_status st = check_book(c, b);
  if (st != GDN_OK) return st;
  if (n_seqs < 0 || total_tokens < 0) return fail(GDN_ERR_ARG, "negative n_seqs/total_tokens");
  if (n_seqs > 65535) return fail(GDN_ERR_SIZE, "n_seqs = %d > 65535", n_seqs);
  if (!cu_seqlens && total_tokens != n_seqs)
    return fail(GDN_ERR_SIZE, "without cu_seqlens total_tokens must equal n_seqs");
  if ((uintptr_t)rows % 8 || ((uintptr_t)positions | (uintptr_t)granted) % 4)
    return fail(GDN_ERR_ARG, "rows must be 8-byte aligned, positions and granted 4-byte");
  if (n_seqs == 0) return ok();
  if (!slot_ids || !pos) return fail(GDN_ERR_ARG, "slot_ids and pos must be non-NULL");
  if (((uintptr_t)slot_ids | (uintptr_t)pos | (uintptr_t)cu_seqlens) % 4)
    return fail(GDN_ERR_ARG, "slot_ids, pos and cu_seqlens must be 4-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->desc.host_checks &&
      ((st = check_host(c, b, slot_ids, pos, "pos", true, cu_seqlens, n_seqs, total_tokens, s)) ||
       (positions && (st = check_device_ptr(positions, "positions"))) ||
       (rows && (st = check_device_ptr(rows, "rows"))) ||
       (granted && (st = check_device_ptr(granted, "granted")))))
    return st;
  const gdn::Book book{b->page_table, b->held, b->free_pages, b->n_free};
  const gdn::SeqIndex seq{slot_ids, cu_seqlens, n_seqs, total_tokens};
  // (a page has 16 tokens at least: the tokens are the larger part)
  const int grid = gdn::grid_for(total_tokens, 2, c->sm_count);
  const cudaError_t e = gdn::kv::launch(gdn::grow_kernel, dim3((unsigned)grid), gdn::kThreads, 0, s,
                                        1, c->view, book, seq, pos, positions, rows, granted);
  if (e != cudaSuccess) return cuda_fail(e, "page growth launch");
  return ok();
}

gdn_status gdn_kv_pages_trim(gdn_kv *c, const gdn_kv_pages *b, const int32_t *slot_ids,
                             const int32_t *lens, int32_t n_seqs, gdn_stream stream) {
  gdn_status st = check_book(c, b);
  if (st != GDN_OK) return st;
  if (n_seqs < 0) return fail(GDN_ERR_ARG, "negative n_seqs");
  if (n_seqs > 65535) return fail(GDN_ERR_SIZE, "n_seqs = %d > 65535", n_seqs);
  if (n_seqs == 0) return ok();
  if (!slot_ids || !lens) return fail(GDN_ERR_ARG, "slot_ids and lens must be non-NULL");
  if (((uintptr_t)slot_ids | (uintptr_t)lens) % 4)
    return fail(GDN_ERR_ARG, "slot_ids and lens must be 4-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c->desc.host_checks &&
      (st = check_host(c, b, slot_ids, lens, "lens", false, nullptr, n_seqs, 0, s)))
    return st;
  const gdn::Book book{b->page_table, b->held, b->free_pages, b->n_free};
  // the most pages that the sequences can hold
  const int64_t most = (int64_t)n_seqs * c->desc.max_pages;
  const int grid = gdn::grid_for(most < c->desc.n_pages ? most : c->desc.n_pages, 8, c->sm_count);
  const cudaError_t e = gdn::kv::launch(gdn::trim_kernel, dim3((unsigned)grid), gdn::kThreads, 0, s,
                                        1, c->view, book, slot_ids, lens, (int)n_seqs);
  if (e != cudaSuccess) return cuda_fail(e, "page trim launch");
  return ok();
}

}  // extern "C"
