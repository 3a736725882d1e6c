// Device helpers of the 8-bit KV cache: scales that are powers of two, and
// codes (int8, or e4m3 floats) to and from float32 and binary16.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "gdn_common.cuh"

namespace gdn {
namespace kv {

// Launch as a programmatic dependent of the kernel before it on the stream: it
// may become resident early, and waits (dependent_wait) before it touches
// global memory until every earlier kernel is complete and visible.  `cluster`:
// CTAs per cluster, along x.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s,
                   int cluster, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Let the next kernel of the stream be set up (it waits for this one itself),
// and wait for those before this one.
__device__ __forceinline__ void dependents_may_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void dependent_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Allow `kernel` `smem` bytes of dynamic shared memory, on its first launch on a
// device (`seen`: the kernel's own, a bit per device; the call costs a launch a
// good part of a microsecond).
template <typename K>
cudaError_t allow_smem(K kernel, int smem, int device, std::atomic<uint64_t> &seen) {
  const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
  if (seen.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) seen.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int CODE>
struct Code;  // top code, exponent range of the scale, conversions

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126..127

// binary16 pairs of two e4m3 codes (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

template <>
struct Code<GDN_KV_I8> {
  static constexpr int kMaxExp = 120;
  // the least e with amax <= 127 * 2^e, in [-100, 120]; amax is finite and >= 0.  With
  // amax = 1.f * 2^(E-127), 127 * 2^(E-133) = 1.984375 * 2^(E-127) covers it unless 1.f is larger.
  static __device__ __forceinline__ int exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 133 + ((b & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    return min(max(e, -100), kMaxExp);
  }
  // y is not NaN
  static __device__ __forceinline__ uint32_t encode(float y) {
    return (uint32_t)__float2int_rn(fminf(fmaxf(y, -127.f), 127.f)) & 0xffu;
  }
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return encode(a) | encode(b) << 8 | encode(c) << 16 | encode(d) << 24;
  }
  static __device__ __forceinline__ float4 decode4(uint32_t w) {
    return make_float4((float)(int8_t)(w & 0xff), (float)(int8_t)(w >> 8 & 0xff),
                       (float)(int8_t)(w >> 16 & 0xff), (float)(int8_t)(w >> 24));
  }
};

template <>
struct Code<GDN_KV_E4M3> {
  static constexpr int kMaxExp = 118;
  // the least e with amax <= 448 * 2^e = 1.75 * 2^(e+8), in [-100, 118]
  static __device__ __forceinline__ int exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, -100), kMaxExp);
  }
  static __device__ __forceinline__ uint32_t encode2(float a, float b) {
    uint16_t r;  // the second operand is the low byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  }
  static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return encode2(a, b) | encode2(c, d) << 16;
  }
  static __device__ __forceinline__ float4 decode4(uint32_t w) {
    const uint32_t lo = e4m3x2_to_half2((uint16_t)(w & 0xffff)), hi = e4m3x2_to_half2((uint16_t)(w >> 16));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

// The exponent of a stored scale: a power of two in the codes' range.  Anything
// else, as in a page that was never written, is brought into it; what is no
// positive finite number counts as the smallest.
template <int CODE>
__device__ __forceinline__ int scale_exponent(float s) {
  const int e = (int)(__float_as_uint(s) >> 23) - 127;  // sign bit set: e > 128
  return e >= 128 ? -100 : min(max(e, -100), Code<CODE>::kMaxExp);
}

// The exponent that a query row is scaled down by, from that of its largest magnitude (128: not
// finite).  Not all of it beyond 116: the row's factor scale * log2(e) * 2^ex has to be finite, and
// binary16 holds the rest.
__device__ __forceinline__ int query_exponent(int ex, bool zero) {
  return ex > 127 || zero ? 0 : min(max(ex, -126), 116);
}

// ---- the softmax's two sums, whose terms may lie further apart than float32 reaches ----
//
// The numerator follows y = x + e (score plus V exponent), the denominator sums 2^(x - M) beside
// it.  Terms of y far below M vanish from the numerator rightly, but a page of small (or all-zero)
// values can have the scores that matter.  So
//   - where a page's exponent is more than kFar below the largest so far, its terms of the
//     denominator come from x - M itself: 2^(y - M) could vanish before 2^-e brings it back;
//   - M is also raised for x + kLowExp, so that no 2^(x - M) is above 2^(15 - kLowExp) and the
//     sum of a whole context stays finite.  The numerator's weights of pages below kLowExp are then
//     up to 2^16 smaller than they could be;
//   - what is carried over to a larger M is scaled in two steps.
constexpr int kLowExp = -84;
constexpr int kFar = 90;

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a * 2^n, n from 127 down to -252 (or -inf): 2^n alone is zero below -126
__device__ __forceinline__ float lower(float a, float n) {
  return a * fast_exp2(fmaxf(n, -126.f)) * fast_exp2(fminf(n + 126.f, 0.f));
}

// The reference of a part that was not computed (those that were have a number or -inf).
__device__ __forceinline__ float no_result() { return __int_as_float(0x7fffffff); }

// A part's sum of the denominator (reference m) under the reference `top` of all parts.  (A part
// without a reference has no weights, or, of a query that is not finite, NaN.)
__device__ __forceinline__ float join_sum(float l, float m, float top) {
  return m == -INFINITY ? l : lower(l, m - top);
}
// The factor of its numerator.
__device__ __forceinline__ float join_factor(float l, float m, float top) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : fast_exp2(m - top);
}

}  // namespace kv
}  // namespace gdn
