// The adapters of a tile of tokens, and rows of bf16 elements.
#pragma once

#include "gdn_adapt.h"
#include "gdn_common.cuh"

namespace gdn {

__device__ __forceinline__ int token_id(const AdaptArgs &g, int t) {
  const int id = t < g.tokens ? g.ids[t] : -1;
  return id >= 0 && id < g.n_adapters ? id : -1;
}

// Elements k .. k + 7 of a row, zeros from `hidden` on (what lies behind a row is not read).  WHOLE:
// hidden is a multiple of 8.
template <bool WHOLE>
__device__ __forceinline__ uint4 load8(const bf16 *row, int k, int hidden) {
  if (WHOLE) return k < hidden ? *reinterpret_cast<const uint4 *>(row + k) : make_uint4(0, 0, 0, 0);
  if (k + 8 <= hidden) return *reinterpret_cast<const uint4 *>(row + k);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (k + j < hidden)
      w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[k + j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One warp: the adapters of tokens tok0 .. tok0 + live - 1 (live <= 256) in the order of their first
// tokens, into list (by lane 0), and their number; kPlanes + 1 if there are more than that.
__device__ __forceinline__ int tile_groups(const AdaptArgs &g, int tok0, int live, int *list) {
  const int lane = threadIdx.x & 31;
  int id[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) id[i] = 32 * i + lane < live ? token_id(g, tok0 + 32 * i + lane) : -1;
  for (int n = 0;; ++n) {
    int first = INT32_MAX, own = -1;  // the first token that is left
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (id[i] >= 0) first = 32 * i + lane, own = id[i];
    const int at = __reduce_min_sync(0xffffffffu, first);
    if (at == INT32_MAX) return n;
    if (n == kPlanes) return n + 1;
    const int next = __shfl_sync(0xffffffffu, own, at & 31);
    if (lane == 0) list[n] = next;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (id[i] == next) id[i] = -1;
  }
}

}  // namespace gdn
