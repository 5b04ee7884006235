// Column sums of partial results, added in a fixed order: the result does not
// depend on which CTA wrote its part first.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

// V columns a thread, 32 V a CTA, a warp for every 32nd part, four of whose
// rows are on their way at once.
template <int V>
__global__ void __launch_bounds__(1024)
colsum_kernel(const ColSum s) {
  __shared__ float red[V][32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int w = blockIdx.y, cols = s.cols[w];
  float *out = s.out[w];
  if (!out || blockIdx.x * 32 * V >= cols) return;
  const int cx = threadIdx.x & 31, py = threadIdx.x >> 5, c = (blockIdx.x * 32 + cx) * V;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.f;
  if (c < cols) {
    const float *from = s.part[w] + c;
    const long long stride = s.stride[w];
#pragma unroll 4
    for (int p = py; p < s.count; p += 32) {
      if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(from + p * stride);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      } else {
        v[0] += from[p * stride];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) red[j][py][cx] = v[j];
  __syncthreads();
  const int co = (blockIdx.x * 32 + py) * V;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float t = warp_sum(red[j][cx][py]);
    if (cx == 0 && co + j < cols) out[co + j] = t;
  }
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
  bool vec = true;  // 16-byte vectors of columns
  for (int i = 0; i < n; ++i)
    vec = vec && (!s.out[i] || (s.cols[i] % 4 == 0 && s.stride[i] % 4 == 0 && reinterpret_cast<uintptr_t>(s.part[i]) % 16 == 0));
  if (vec && most >= 4096)
    return launch_k(colsum_kernel<4>, dim3((most + 127) / 128, n), dim3(1024), 0, st, true, s);
  return launch_k(colsum_kernel<1>, dim3((most + 31) / 32, n), dim3(1024), 0, st, true, s);
}

}  // namespace ret
