// Column sums of partial results, added in a fixed order: the result does not
// depend on which CTA wrote its part first.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

// 32 columns a CTA, a warp for every 32nd part.
__global__ void __launch_bounds__(1024)
colsum_kernel(const ColSum s) {
  __shared__ float red[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int w = blockIdx.y, cols = s.cols[w];
  float *out = s.out[w];
  if (!out || blockIdx.x * 32 >= cols) return;
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
  float v = 0.f;
  if (c < cols)
    for (int p = py; p < s.count; p += 32) v += s.part[w][p * s.stride[w] + c];
  red[py][cx] = v;
  __syncthreads();
  v = warp_sum(red[cx][py]);
  const int co = blockIdx.x * 32 + py;
  if (cx == 0 && co < cols) out[co] = v;
}

}  // namespace

cudaError_t launch_colsum(const ColSum &s, cudaStream_t st) {
  int most = 0, n = 0;
  for (int i = 0; i < 3; ++i)
    if (s.out[i]) {
      most = std::max(most, s.cols[i]);
      n = i + 1;
    }
  if (most == 0) return cudaSuccess;
  return launch_k(colsum_kernel, dim3((most + 31) / 32, n), dim3(1024), 0, st, true, s);
}

}  // namespace ret
