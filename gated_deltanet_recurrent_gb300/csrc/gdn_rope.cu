// Rotary positions on query and key heads: the first `rot` elements of every head are pairs
// (a, b), turned by the angle p * theta_j of the token's position p and the pair's j:
//     a' = s (a cos - b sin),   b' = s (b cos + a sin).
//
// The angle is formed in turns and in whole numbers: theta_j / 2 pi is held as a 64-bit binary
// fraction f_j, and p * f_j modulo 2^64 -- one wrapping product -- is the angle modulo a turn, off by
// 2^-65 p and by p times what theta_j, a 64-bit float, is off by (2^-53 of it and a few more).  So the
// product takes no 64-bit floats, whose rate here is a sixtieth of the 32-bit one.  Its upper 24 bits go to sincospi, the rest is a first-order
// correction, so that sine and cosine are as good as their rounding to float32.
//
// HBM-bound: each head is read once and written once.  A CTA takes up to four tokens: it asks for the
// first elements, computes the tokens' sines and cosines once into shared memory while they come
// (all heads of a token share them), and turns head after head, two a thread in flight.  A thread
// keeps its place within the head, so that nothing is divided.  Measured: 16384 tokens of 16 + 2 heads
// of 256, 64 elements turned, the rest copied (302 MB), 53 us, 5.7 TB/s; 5003 float32 tokens of 28 + 4
// heads of 128 (164 MB) 26 us, 6.3 TB/s.  (Eight tokens a CTA and one head in flight: 63 and 31 us;
// eight and four 58 and 31; two tokens and four heads 61 and 27.)
#include <cmath>
#include <new>

#include "gdn_common.cuh"
#include "gdn_host.h"
#include "gdn_kv.cuh"

namespace gdn {
namespace {

constexpr int kMaxPairs = 256;   // rot <= 512
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // tokens per CTA, at most
constexpr int kAhead = 2;        // heads that a thread has in flight

// theta_j / 2 pi as 64-bit fractions of a turn
struct Turns {
  uint64_t f[kMaxPairs];
};

struct RopeArgs {
  const int32_t *positions;
  const void *x[2];        // q, k
  void *y[2];
  int64_t ld_x[2], ld_y[2];
  int heads[2];
  int tokens, d, pairs;    // pairs = rot / 2
  int copies;              // 1: elements behind the pairs are copied, 0: they are in place
  float scale;
};

__device__ __forceinline__ float2 turned(uint64_t t, float scale) {
  const int32_t hi = (int32_t)(t >> 32) & ~0xff;               // 24 bits: exact in float32
  const float x = (float)hi * 0x1p-31f;                        // half turns, in [-1, 1)
  const float rest = (float)(uint32_t)(t >> 8) * 0x1p-32f;     // of the lowest bit of hi, in [0, 1]
  const float r = rest * (0x1p-23f * 3.14159265f);             // radians
  float s, c;
  sincospif(x, &s, &c);
  // (the second order is below 2^-43)
  return make_float2((c - r * s) * scale, (s + r * c) * scale);
}

// V elements, moved as one word; SPLIT: one by one, where they are aligned to nothing more.
template <typename T, int V, bool SPLIT>
struct Vec {
  static constexpr int kBytes = V * (int)sizeof(T);
  using Raw = std::conditional_t<
      kBytes == 16, uint4,
      std::conditional_t<kBytes == 8, uint2, std::conditional_t<kBytes == 4, uint32_t, uint16_t>>>;
  union U {
    Raw raw;
    T e[V];
    __device__ U() {}
  };
  static __device__ __forceinline__ Raw load(const T *p) {
    if constexpr (!SPLIT) return *reinterpret_cast<const Raw *>(p);
    U u;
#pragma unroll
    for (int j = 0; j < V; ++j) u.e[j] = p[j];
    return u.raw;
  }
  static __device__ __forceinline__ void store(T *p, Raw r) {
    if constexpr (!SPLIT) {
      *reinterpret_cast<Raw *>(p) = r;
    } else {
      U u;
      u.raw = r;
#pragma unroll
      for (int j = 0; j < V; ++j) p[j] = u.e[j];
    }
  }
  static __device__ __forceinline__ void widen(Raw r, float *x) {
    U u;
    u.raw = r;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = Elem<T>::load1(&u.e[j]);
  }
  static __device__ __forceinline__ Raw narrow(const float *x) {
    U u;
#pragma unroll
    for (int j = 0; j < V; ++j) Elem<T>::store1(&u.e[j], x[j]);
    return u.raw;
  }
};

// Two vectors of V elements that belong together: the a's and b's of V pairs (half layout), or V
// elements of neighbouring pairs and nothing (interleaved; copies).
template <typename T, int V, bool HALF, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ Turns turns, const __grid_constant__ RopeArgs a,
                int per_cta) {
  using X = Vec<T, V, SPLIT>;
  constexpr int U = kAhead;
  extern __shared__ float2 s_turn[];  // [per_cta][pairs]
  kv::dependents_may_launch();
  kv::dependent_wait();
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  const int tok0 = blockIdx.x * per_cta, n_tok = min(per_cta, a.tokens - tok0);
  const int heads = a.heads[0] + a.heads[1];
  // places within a head: pairs first, then what is copied; a thread's place changes only when its
  // tokens are done (w), and it goes through them head by head (t, h)
  const int turning = HALF ? a.pairs / V : 2 * a.pairs / V;
  const int places = turning + (a.copies ? (a.d - 2 * a.pairs) / V : 0);
  const int dt = blockDim.y / heads, dh = blockDim.y - dt * heads;
  const int t0 = threadIdx.y / heads, h0 = threadIdx.y - t0 * heads;
  int w = threadIdx.x, t = t0, h = h0;
  typename X::Raw r[U], v[U];
  T *y[U];
  int cs[U];  // the place's first sine, -1: a copy, -2: nothing
  auto load = [&]() {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      cs[i] = -2;
      if (t >= n_tok) {
        w += blockDim.x;
        t = t0, h = h0;
      }
      if (w >= places || t >= n_tok) continue;
      const bool turn = w < turning;
      const int at = turn ? w * V : 2 * a.pairs + (w - turning) * V;
      const int side = h >= a.heads[0], hh = side ? h - a.heads[0] : h;
      const int64_t off = (int64_t)hh * a.d + at;
      const T *x = static_cast<const T *>(a.x[side]) + (tok0 + t) * a.ld_x[side] + off;
      y[i] = static_cast<T *>(a.y[side]) + (tok0 + t) * a.ld_y[side] + off;
      cs[i] = turn ? t * a.pairs + (HALF ? at : at / 2) : -1;
      r[i] = X::load(x);
      if (HALF && turn) v[i] = X::load(x + a.pairs);
      h += dh;
      t += dt;
      if (h >= heads) h -= heads, ++t;
    }
  };
  load();  // on their way while the angles are computed
  for (int i = tid; i < n_tok * a.pairs; i += threads) {
    const int tt = i / a.pairs, j = i - tt * a.pairs;
    const int64_t p = a.positions[tok0 + tt];
    s_turn[i] = turned((uint64_t)p * turns.f[j], a.scale);
  }
  __syncthreads();
  while (cs[0] != -2) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (cs[i] == -2) continue;
      if (cs[i] >= 0) {
        const float2 *turn = s_turn + cs[i];
        float u[V];
        X::widen(r[i], u);
        if constexpr (HALF) {
          float z[V], yu[V], yv[V];
          X::widen(v[i], z);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            yu[e] = u[e] * turn[e].x - z[e] * turn[e].y;
            yv[e] = z[e] * turn[e].x + u[e] * turn[e].y;
          }
          r[i] = X::narrow(yu);
          X::store(y[i] + a.pairs, X::narrow(yv));
        } else {
          float yu[V];
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            yu[e] = u[e] * turn[e / 2].x - u[e + 1] * turn[e / 2].y;
            yu[e + 1] = u[e + 1] * turn[e / 2].x + u[e] * turn[e / 2].y;
          }
          r[i] = X::narrow(yu);
        }
      }
      X::store(y[i], r[i]);
    }
    load();
  }
}

template <typename T, int V, bool HALF, bool SPLIT = false>
cudaError_t launch(const Turns &f, const RopeArgs &a, cudaStream_t s) {
  const int places = (HALF ? a.pairs / V : 2 * a.pairs / V) +
                     (a.copies ? (a.d - 2 * a.pairs) / V : 0);
  const int x = places < kRopeThreads ? places : kRopeThreads;
  // (few tokens: a CTA each, for the latency)
  const int per_cta = a.tokens >= 1024 * kRopeTokens ? kRopeTokens : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.tokens + per_cta - 1) / per_cta));
  cfg.blockDim = dim3((unsigned)x, (unsigned)(kRopeThreads / x));
  cfg.dynamicSmemBytes = sizeof(float2) * per_cta * a.pairs;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<T, V, HALF, SPLIT>, f, a, per_cta);
}

template <typename T, bool HALF>
cudaError_t launch_v(const Turns &f, const RopeArgs &a, int v, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (v == 8) return launch<T, 8, HALF>(f, a, s);
  if (v >= 4) return launch<T, 4, HALF>(f, a, s);
  if (v >= 2) return launch<T, 2, HALF>(f, a, s);
  if constexpr (HALF)
    return launch<T, 1, true>(f, a, s);
  else  // both elements of a pair are one thread's
    return launch<T, 2, false, true>(f, a, s);
}

}  // namespace
}  // namespace gdn

struct gdn_rope_plan {
  gdn_rope_desc desc;
  gdn::Turns turns;
};

namespace {

using namespace gdn::host;

constexpr double kPi = 3.14159265358979323846;

gdn_status check_desc(const gdn_rope_desc *r) {
  if (!r) return fail(GDN_ERR_ARG, "desc is NULL");
  if (r->d % 2 || r->rot < 2 || r->rot % 2 || r->rot > r->d)
    return fail(GDN_ERR_ARG, "d (%d) must be even, and rot (%d) even and within 2 .. d", r->d,
                r->rot);
  if (r->rot > 2 * gdn::kMaxPairs || r->d > 4096)
    return fail(GDN_ERR_UNSUPPORTED, "rot = %d, d = %d (at most %d and 4096)", r->rot, r->d,
                2 * gdn::kMaxPairs);
  if (r->layout != GDN_ROPE_HALF && r->layout != GDN_ROPE_INTERLEAVED)
    return fail(GDN_ERR_ARG, "layout must be GDN_ROPE_HALF or GDN_ROPE_INTERLEAVED");
  if (!(r->base > 0) || !std::isfinite(r->base))
    return fail(GDN_ERR_ARG, "base must be positive and finite");
  if (!(r->factor > 0) || !std::isfinite(r->factor))
    return fail(GDN_ERR_ARG, "factor must be positive and finite");
  if (r->original_len < 0) return fail(GDN_ERR_ARG, "original_len is negative");
  if (r->original_len > 0 && (!(r->low_turns >= 0) || !(r->high_turns > r->low_turns) ||
                              !std::isfinite(r->high_turns)))
    return fail(GDN_ERR_ARG, "0 <= low_turns < high_turns needed with original_len");
  if (!std::isfinite(r->out_scale)) return fail(GDN_ERR_ARG, "out_scale is not finite");
  return GDN_OK;
}

// theta_j / 2 pi modulo one, as a 64-bit fraction: whole turns change nothing.
uint64_t fraction(double turns) {
  double x = std::floor(turns);
  x = turns - x;                               // [0, 1)
  const double hi = std::floor(std::ldexp(x, 32));
  const double lo = std::ldexp(std::ldexp(x, 32) - hi, 32);
  return ((uint64_t)hi << 32) + (uint64_t)std::llround(lo);
}

// Elements per vector: as many as every row, head and border within the head allows.
int vector_elements(const gdn_rope_desc &r, const gdn::RopeArgs &a, size_t es) {
  int v = (int)(16 / es);
  const int border = r.layout == GDN_ROPE_HALF ? r.rot / 2 : r.rot;
  auto fits = [&](int64_t n) { return n % v == 0; };
  for (; v > 1; v /= 2) {
    bool good = fits(border) && fits(r.d);
    for (int i = 0; i < 2 && good; ++i)
      if (a.heads[i])
        good = fits(a.ld_x[i]) && fits(a.ld_y[i]) && (uintptr_t)a.x[i] % (v * es) == 0 &&
               (uintptr_t)a.y[i] % (v * es) == 0;
    if (good) break;
  }
  return v;
}

}  // namespace

extern "C" {

gdn_status gdn_rope_create(const gdn_rope_desc *desc, gdn_rope_plan **out) {
  if (!out) return fail(GDN_ERR_ARG, "out is NULL");
  *out = nullptr;
  const gdn_status st = check_desc(desc);
  if (st != GDN_OK) return st;
  gdn_rope_plan *p = new (std::nothrow) gdn_rope_plan;
  if (!p) return fail(GDN_ERR_SIZE, "no host memory for the handle");
  p->desc = *desc;
  for (int j = 0; j < gdn::kMaxPairs; ++j) p->turns.f[j] = 0;
  for (int j = 0; j < desc->rot / 2; ++j) {
    double theta = std::pow(desc->base, -2.0 * j / desc->rot);
    if (desc->original_len > 0) {
      const double turns = theta * (double)desc->original_len / (2 * kPi);
      double keep = (turns - desc->low_turns) / (desc->high_turns - desc->low_turns);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      theta *= keep + (1 - keep) / desc->factor;
    } else {
      theta /= desc->factor;
    }
    if (!std::isfinite(theta)) {
      delete p;
      return fail(GDN_ERR_ARG, "the frequency of pair %d is not finite", j);
    }
    p->turns.f[j] = fraction(theta / (2 * kPi));
  }
  *out = p;
  return ok();
}

gdn_status gdn_rope_destroy(gdn_rope_plan *p) {
  delete p;
  return ok();
}

gdn_status gdn_rope(const gdn_rope_plan *p, int32_t tokens, const int32_t *positions, const void *q,
                    int64_t ld_q, int32_t h_q, const void *k, int64_t ld_k, int32_t h_k,
                    void *q_out, int64_t ld_q_out, void *k_out, int64_t ld_k_out, gdn_dtype dtype,
                    gdn_stream stream) {
  if (!p) return fail(GDN_ERR_ARG, "plan is NULL");
  if (tokens < 0 || h_q < 0 || h_k < 0) return fail(GDN_ERR_ARG, "negative tokens or heads");
  if (!dtype_ok(dtype)) return fail(GDN_ERR_DTYPE, "dtype must be F32 or BF16");
  if (h_q > 65535 || h_k > 65535) return fail(GDN_ERR_UNSUPPORTED, "more than 65535 heads");
  const gdn_rope_desc &r = p->desc;
  const size_t es = dtype_size(dtype);
  if (tokens == 0 || h_q + h_k == 0) return ok();
  if (!positions) return fail(GDN_ERR_ARG, "positions is NULL");
  if ((uintptr_t)positions % 4) return fail(GDN_ERR_ARG, "positions must be 4-byte aligned");
  gdn::RopeArgs a = {positions, {q, k}, {q_out, k_out}, {ld_q, ld_k}, {ld_q_out, ld_k_out},
                     {h_q, h_k}, tokens, r.d, r.rot / 2, 0, r.out_scale};
  gdn_status st;
  if (r.host_checks && (st = check_device_ptr(positions, "positions"))) return st;
  for (int i = 0; i < 2; ++i) {
    const char *name = i ? "k" : "q";
    if (a.heads[i] == 0) continue;
    if (!a.x[i] || !a.y[i]) return fail(GDN_ERR_ARG, "%s and %s_out must be non-NULL", name, name);
    const int64_t width = (int64_t)a.heads[i] * r.d;
    if (a.ld_x[i] == 0) a.ld_x[i] = width;
    if (a.ld_y[i] == 0) a.ld_y[i] = width;
    if (a.ld_x[i] < width || a.ld_y[i] < width)
      return fail(GDN_ERR_ARG, "%s: token stride smaller than a token", name);
    if ((uintptr_t)a.x[i] % es || (uintptr_t)a.y[i] % es)
      return fail(GDN_ERR_ARG, "%s is not aligned to its elements", name);
    if (a.x[i] != a.y[i])
      a.copies = 1;
    else if (a.ld_x[i] != a.ld_y[i] && tokens > 1)
      return fail(GDN_ERR_ARG, "%s in place needs one token stride", name);
    if (r.host_checks && ((st = check_device_ptr(a.x[i], name)) || (st = check_device_ptr(a.y[i], name))))
      return st;
  }
  if (r.rot == r.d) a.copies = 0;
  const int v = vector_elements(r, a, es);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = r.layout == GDN_ROPE_HALF;
  const cudaError_t e =
      dtype == GDN_F32
          ? half ? gdn::launch_v<float, true>(p->turns, a, v, s)
                 : gdn::launch_v<float, false>(p->turns, a, v, s)
          : half ? gdn::launch_v<gdn::bf16, true>(p->turns, a, v, s)
                 : gdn::launch_v<gdn::bf16, false>(p->turns, a, v, s);
  if (e != cudaSuccess) return cuda_fail(e, "rotary launch");
  return ok();
}

}  // extern "C"
