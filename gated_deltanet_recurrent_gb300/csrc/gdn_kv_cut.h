// How the split attention kernel cuts its line of tiles among the CTAs (plain
// arithmetic, for the device and for host code).
#pragma once

#include "gdn_internal.h"

namespace gdn {

// a * b / c, in 32 bits where they are enough for the product and for c
GDN_HD int64_t mul_div(int64_t a, int64_t b, int64_t c) {
  const int64_t x = a * b;
  return (x | c) >> 32 == 0 ? (int64_t)((uint32_t)x / (uint32_t)c) : x / c;
}

// How the line of tiles is cut: segments (one, or one for each order of a CTA
// on its SM, by share), each into equal pieces.
template <typename Cfg>
struct Cut {
  int64_t total;
  int per, segments;  // CTAs of a segment
  GDN_HD int64_t segment(int o) const {
    if (segments == 1) return o ? total : 0;
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < Cfg::kCtas; ++i) {
      if (i < o) before += Cfg::kShare(i);
      all += Cfg::kShare(i);
    }
    return total * before / all;
  }
  // first tile of CTA i's piece
  GDN_HD int64_t begin(int i) const {
    const int o = i / per;
    const int64_t from = segment(o);
    return o == segments ? from : from + mul_div(segment(o + 1) - from, i - o * per, per);
  }
  // the CTA whose piece holds tile x
  GDN_HD int owner(int64_t x) const {
    int o = 0;
    while (o + 1 < segments && segment(o + 1) <= x) ++o;
    const int64_t from = segment(o), len = segment(o + 1) - from;
    return o * per + (int)mul_div(x - from + 1, per, len) -
           ((x - from + 1) * per % len == 0 ? 1 : 0);
  }
};

}  // namespace gdn
