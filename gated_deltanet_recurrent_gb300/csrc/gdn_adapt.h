// What the projection with adapters needs: shared by its entry point and its kernels.
#pragma once

#include "gdn_internal.h"

namespace gdn {

struct AdaptArgs {
  const void *x, *w, *a, *b;  // bf16: x [tokens][hidden], w [n_out][hidden], a [n_adapters][rank]
                              // [hidden], b [n_adapters][n_out][rank]
  const float *scale;         // [n_adapters]
  const int32_t *ids;         // [tokens]
  void *y;                    // [tokens][n_out]
  int64_t ld_x, ld_w, ld_a, ld_b, ld_y;
  int tokens, hidden, n_out, rank, n_adapters;
  gdn_dtype y_dtype;
  // workspace: scale * A x in bf16 parts that add up to it, [parts][tokens][rank_pad], zeros beyond
  // rank; with tile > 0 [kPlanes][parts][tokens][rank_pad]: of a tile of `tile` tokens with n <=
  // kPlanes adapters, plane j < n has the h of the j-th adapter's tokens (in the order of their
  // first ones) and zeros for the others; with more, plane 0 has all h there is
  void *h;
  int tile;
  unsigned int *err;
  int sm_count, device;
  uint32_t test_flags;  // GDN_TEST_ADAPT_* bits of the pool; 0 in normal use
  GDN_HD int parts() const { return y_dtype == GDN_F32 ? 3 : 2; }
  // the rank rounded up to the tensor cores' 16
  GDN_HD int rank16() const { return (rank + 15) & ~15; }
  // and to the width of the rows that the projection reads
  GDN_HD int rank_pad() const { return rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
};

// (With 64, 512 tokens with 64 adapters, 2048 -> 5120 at rank 64, took 140 us, with eight 112.)
constexpr int kPlanes = 8;

size_t adapt_workspace_bytes(const AdaptArgs &g);
// The `tile` that the kernels of this call go by.
int adapt_tile(const AdaptArgs &g);
// The low side, then the projection; cudaErrorNotSupported: no tensor map.
cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t s);

// The projection of many tokens, on pairs of CTAs.
cudaError_t launch_adapt_pair(const AdaptArgs &g, cudaStream_t s);

// others: CTAs of the projection that want an SM while the low side has its own.
cudaError_t launch_adapt_low(const AdaptArgs &g, int others, cudaStream_t s);

}  // namespace gdn
