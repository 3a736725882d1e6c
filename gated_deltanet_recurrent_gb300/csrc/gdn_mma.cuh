// mma.sync for products whose operands come from global memory straight into registers.
#pragma once

#include <stdint.h>

namespace gdn {

// d (16 x 8) += a (16 x 16) b (16 x 8), bf16, float32 sums.  Lane (r, c) = (lane / 4, lane % 4): a has
// rows r, r + 8 and two K places of two elements each, a[0], a[1] the first and a[2], a[3] the second;
// b0, b1 are column r at the same places; d[0], d[1] is row r, columns 2 c and 2 c + 1, d[2], d[3] row
// r + 8.
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace gdn
