// The input projection with a low-rank adapter per token:
//     y[t] = W x[t] + c[a] B[a] (A[a] x[t]),   a = ids[t]   (W x[t] alone where ids[t] = -1).
//
// Two kernels: the low side h[t] = c[a] A[a] x[t] in float32, then the projection, whose tiles add
// B[a] h[t] before y is rounded once.
#include "gdn_adapt.h"
#include "gdn_common.cuh"

namespace gdn {
namespace {

// h[t][r]: a warp per token and rank
__global__ void low_kernel(AdaptArgs g) {
  const int64_t unit = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (unit >= (int64_t)g.tokens * g.rank) return;
  const int t = (int)(unit / g.rank), r = (int)(unit % g.rank);
  const int id = g.ids[t];
  if (id < 0 || id >= g.n_adapters) {
    if (id != -1 && r + lane == 0) raise_error(g.err, GDN_DEVERR_ADAPTER);
    return;
  }
  const bf16 *x = static_cast<const bf16 *>(g.x) + t * g.ld_x;
  const bf16 *a = static_cast<const bf16 *>(g.a) + ((int64_t)id * g.rank + r) * g.ld_a;
  float sum = 0.f;
  for (int k = lane; k < g.hidden; k += 32) sum += __bfloat162float(x[k]) * __bfloat162float(a[k]);
  sum = group_sum<32>(sum);
  if (lane == 0) g.h[(int64_t)t * g.rank + r] = sum * g.scale[id];
}

// 64 x 64 outputs a CTA, 4 x 4 a thread
template <typename TO>
__global__ void __launch_bounds__(256) project_kernel(AdaptArgs g) {
  __shared__ float s_x[16][65], s_w[16][65];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t t0 = (int64_t)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.hidden; k0 += 16) {
    for (int i = tid; i < 64 * 16; i += 256) {
      const int row = i >> 4, k = k0 + (i & 15);
      const bool in = k < g.hidden;
      s_x[i & 15][row] = in && t0 + row < g.tokens
          ? __bfloat162float(static_cast<const bf16 *>(g.x)[(t0 + row) * g.ld_x + k]) : 0.f;
      s_w[i & 15][row] = in && n0 + row < g.n_out
          ? __bfloat162float(static_cast<const bf16 *>(g.w)[(n0 + row) * g.ld_w + k]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += s_x[k][ty + 16 * i] * s_w[k][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty + 16 * i;
    if (t >= g.tokens) continue;
    const int id = g.ids[t];
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx + 16 * j;
      if (n >= g.n_out) continue;
      float v = acc[i][j];
      if (id >= 0 && id < g.n_adapters) {
        const bf16 *b = static_cast<const bf16 *>(g.b) + ((int64_t)id * g.n_out + n) * g.ld_b;
        float d = 0.f;
        for (int r = 0; r < g.rank; ++r) d += g.h[t * g.rank + r] * __bfloat162float(b[r]);
        v += d;
      }
      Elem<TO>::store1(static_cast<TO *>(g.y) + t * g.ld_y + n, v);
    }
  }
}

}  // namespace

size_t adapt_workspace_bytes(const AdaptArgs &g) { return (size_t)g.tokens * g.rank * 4; }

cudaError_t launch_adapt(const AdaptArgs &g, cudaStream_t s) {
  const int64_t warps = (int64_t)g.tokens * g.rank;
  low_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((g.n_out + 63) / 64), (unsigned)((g.tokens + 63) / 64));
  if (g.y_dtype == GDN_F32)
    project_kernel<float><<<grid, 256, 0, s>>>(g);
  else
    project_kernel<bf16><<<grid, 256, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace gdn
