// Column sums of partial results, added in a fixed order: the result does not
// depend on which CTA wrote its part first.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

// V columns a thread, 32 V a CTA, every P-th part a thread, eight of them on
// their way at once (256 parts of 65536 columns 25 us, 2.7 TB/s; 1024 of 16384
// eight at a time 48, 32 at a time 28).
template <int V, int P>
__global__ void __launch_bounds__(32 * P)
colsum_kernel(const ColSum s) {
  __shared__ float red[V][P][33];
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
#pragma unroll 8
    for (int p = py; p < s.count; p += P) {
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
  for (int i = threadIdx.x; i < 32 * V; i += 32 * P) {
    const int col = blockIdx.x * 32 * V + i;
    float t = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) t += red[i % V][p][i / V];
    if (col < cols) out[col] = t;
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
  // Vectors of columns where they are there and enough; eight parts at a time
  // where those are few or the columns fill the SMs, else 32.
  const bool many = s.count > 128;
  if (vec && most >= 16384) {
    const dim3 grid((most + 127) / 128, n);
    if (many && most < 128 * 4 * device_sms()) return launch_k(colsum_kernel<4, 32>, grid, dim3(1024), 0, st, true, s);
    return launch_k(colsum_kernel<4, 8>, grid, dim3(256), 0, st, true, s);
  }
  const dim3 grid((most + 31) / 32, n);
  if (many) return launch_k(colsum_kernel<1, 32>, grid, dim3(1024), 0, st, true, s);
  return launch_k(colsum_kernel<1, 8>, grid, dim3(256), 0, st, true, s);
}

}  // namespace ret
