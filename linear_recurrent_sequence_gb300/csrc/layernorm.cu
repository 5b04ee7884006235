// LayerNorm over rows of d values and its gradients.
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps), biased variance;
//   with h = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum_rows dy h,  db = sum_rows dy.
// fp32 arithmetic for bf16 and fp32 rows; mean, rstd, w, b, dw, db in fp32.
// Both directions are bound by memory: 2 (forward) or 3 (backward) row
// elements move per value and at most 13 flop are done with them.
//
// The variance is the mean square of the deviations, taken after the mean:
// a row with a large level loses nothing to cancellation.
#include <algorithm>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

constexpr int kMaxWarps = 32;

// Sums of N values over the threads that share a row: one warp, or the CTA
// through red (one barrier; consecutive calls alternate between two
// buffers, so a warp that is ahead cannot overwrite what another still reads).
template <int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*red)[kMaxWarps], bool one_warp) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
  if (one_warp) return;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][w] = x[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(lane < nw ? red[i][lane] : 0.f);
}

// One row per CTA of up to 1024 threads, NV vectors of VEC values a thread,
// the row in registers between the three uses of it.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
ln_fwd_kernel(const LnArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  const bool one_warp = blockDim.x == 32;
  const int step = blockDim.x * VEC, t0 = threadIdx.x * VEC;
  const float inv_d = 1.f / (float)a.d;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    T *y = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
    float v[NV][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t0 + i * step;
      if (c < a.d) {
        Elems<T, VEC> e;
        e.load(x + c);
        e.get(v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0] += v[i][j];
    }
    row_sums<1>(s, red[0], one_warp);
    const float mean = s[0] * inv_d;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t0 + i * step < a.d)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] -= mean;
          q[0] = fmaf(v[i][j], v[i][j], q[0]);
        }
    row_sums<1>(q, red[1], one_warp);
    const float rstd = rsqrtf(fmaf(q[0], inv_d, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t0 + i * step;
      if (c < a.d) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = v[i][j] * rstd;
          const float g = a.w ? a.w[c + j] : 1.f;
          o[j] = a.b ? fmaf(h, g, a.b[c + j]) : h * g;
        }
        Elems<T, VEC> e;
        e.set(o);
        e.store(y + c);
      }
    }
  }
}

// Rows too long for registers: the row is read three times (the second and
// third reading come from the caches).
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
ln_fwd_long_kernel(const LnArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int step = blockDim.x * VEC, t0 = threadIdx.x * VEC;
  const float inv_d = 1.f / (float)a.d;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    T *y = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
    float s[1] = {0.f}, q[1] = {0.f};
    Elems<T, VEC> e;
    float v[VEC];
    for (int c = t0; c < a.d; c += step) {
      e.load(x + c);
      e.get(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[0] += v[j];
    }
    row_sums<1>(s, red[0], false);
    const float mean = s[0] * inv_d;
    for (int c = t0; c < a.d; c += step) {
      e.load(x + c);
      e.get(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[0] = fmaf(v[j] - mean, v[j] - mean, q[0]);
    }
    row_sums<1>(q, red[1], false);
    const float rstd = rsqrtf(fmaf(q[0], inv_d, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    for (int c = t0; c < a.d; c += step) {
      e.load(x + c);
      e.get(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = (v[j] - mean) * rstd;
        const float g = a.w ? a.w[c + j] : 1.f;
        v[j] = a.b ? fmaf(h, g, a.b[c + j]) : h * g;
      }
      e.set(v);
      e.store(y + c);
    }
  }
}

// dx of the CTA's rows, and the sums of dy h and dy over them: each thread
// keeps the sums of its own NV x VEC columns in registers and writes them to
// part[blockIdx][2][d] once at the end.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(1024)
ln_bwd_kernel(const LnArgs a, float *__restrict__ part) {
  __shared__ float red[2][2][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  const bool one_warp = blockDim.x == 32;
  const int step = blockDim.x * VEC, t0 = threadIdx.x * VEC;
  const float inv_d = 1.f / (float)a.d;
  float aw[NV][VEC], ab[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) aw[i][j] = ab[i][j] = 0.f;
  int par = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, par ^= 1) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    const T *dy = reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r);
    T *dx = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
    const float mean = a.mean[r], rstd = a.rstd[r];
    float h[NV][VEC], g[NV][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t0 + i * step;
      if (c < a.d) {
        Elems<T, VEC> ex, eg;
        ex.load(x + c);
        eg.load(dy + c);
        ex.get(h[i]);
        eg.get(g[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[i][j] = (h[i][j] - mean) * rstd;
          aw[i][j] = fmaf(g[i][j], h[i][j], aw[i][j]);
          ab[i][j] += g[i][j];
          if (a.w) g[i][j] *= a.w[c + j];
          s[0] += g[i][j];
          s[1] = fmaf(g[i][j], h[i][j], s[1]);
        }
      }
    }
    row_sums<2>(s, red[par], one_warp);
    const float c1 = s[0] * inv_d, c2 = s[1] * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t0 + i * step;
      if (c < a.d) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[i][j] = rstd * (g[i][j] - fmaf(h[i][j], c2, c1));
        Elems<T, VEC> e;
        e.set(g[i]);
        e.store(dx + c);
      }
    }
  }
  if (!part) return;
  float *pw = part + (size_t)blockIdx.x * 2 * a.d, *pb = pw + a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t0 + i * step;
    if (c < a.d)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        pw[c + j] = aw[i][j];
        pb[c + j] = ab[i][j];
      }
  }
}

// Rows too long for one CTA's registers, in two passes: mean(g) and
// mean(g h) of each row (stat[r][2]), then dx and the column sums by column
// blocks.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
ln_bwd_stat_kernel(const LnArgs a, float *__restrict__ stat) {
  __shared__ float red[2][2][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  int par = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, par ^= 1) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    const T *dy = reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r);
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x * VEC; c < a.d; c += blockDim.x * VEC) {
      Elems<T, VEC> ex, eg;
      ex.load(x + c);
      eg.load(dy + c);
      float h[VEC], g[VEC];
      ex.get(h);
      eg.get(g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (a.w) g[j] *= a.w[c + j];
        s[0] += g[j];
        s[1] = fmaf(g[j], (h[j] - mean) * rstd, s[1]);
      }
    }
    row_sums<2>(s, red[par], false);
    if (threadIdx.x < 2) stat[2 * r + threadIdx.x] = s[threadIdx.x] / (float)a.d;
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256)
ln_bwd_cols_kernel(const LnArgs a, const float *__restrict__ stat, float *__restrict__ part) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * VEC;
  if (c >= a.d) return;
  float aw[VEC], ab[VEC], w[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    aw[j] = ab[j] = 0.f;
    w[j] = a.w ? a.w[c + j] : 1.f;
  }
  for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float mean = a.mean[r], rstd = a.rstd[r], c1 = stat[2 * r], c2 = stat[2 * r + 1];
    Elems<T, VEC> ex, eg;
    ex.load(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r) + c);
    eg.load(reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r) + c);
    float h[VEC], g[VEC];
    ex.get(h);
    eg.get(g);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      h[j] = (h[j] - mean) * rstd;
      aw[j] = fmaf(g[j], h[j], aw[j]);
      ab[j] += g[j];
      g[j] = rstd * (g[j] * w[j] - fmaf(h[j], c2, c1));
    }
    eg.set(g);
    eg.store(reinterpret_cast<T *>(a.out) + row_offset(a.so, r) + c);
  }
  if (!part) return;
  float *pw = part + (size_t)blockIdx.y * 2 * a.d, *pb = pw + a.d;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    pw[c + j] = aw[j];
    pb[c + j] = ab[j];
  }
}

// dw, db = the sums of the G partial rows, in a fixed order: the result does
// not depend on which CTA finished first.
__global__ void __launch_bounds__(1024)
ln_bwd_sum_kernel(const float *__restrict__ part, int G, int d, float *__restrict__ dw,
                  float *__restrict__ db) {
  __shared__ float red[32][33];
  pdl_launch_dependents();
  pdl_wait();
  float *out = blockIdx.y ? db : dw;
  if (!out) return;
  const int cx = threadIdx.x & 31, gy = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
  float s = 0.f;
  if (c < d)
    for (int g = gy; g < G; g += 32) s += part[((size_t)g * 2 + blockIdx.y) * d + c];
  red[gy][cx] = s;
  __syncthreads();
  s = warp_sum(red[cx][gy]);
  const int co = blockIdx.x * 32 + gy;
  if (cx == 0 && co < d) out[co] = s;
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return 1;
  return sms;
}

// 16-byte vectors need every row of every operand on a 16-byte boundary.
bool rows_aligned(const void *p, const RowSet &s, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (s.n1 == 1 || s.s1 * esz % 16 == 0) &&
         (s.n0 == 1 || s.s0 * esz % 16 == 0);
}

int threads_for(int d, int per_thread, int most) {
  const int t = (d + per_thread - 1) / per_thread;
  const int r = (t + 31) / 32 * 32;
  return r > most ? most : r;
}

template <typename T, int VEC, int NV>
cudaError_t fwd(const LnArgs &a, cudaStream_t st) {
  const long long cap = 1LL << 30;
  return launch_k(ln_fwd_kernel<T, VEC, NV>, dim3((unsigned)(a.rows < cap ? a.rows : cap)),
                  dim3(threads_for(a.d, VEC * NV, 1024)), 0, st, true, a);
}

template <typename T, int VEC>
cudaError_t fwd_any(const LnArgs &a, cudaStream_t st) {
  if (a.d <= 512 * VEC) return fwd<T, VEC, 1>(a, st);
  if (a.d <= 2048 * VEC) return fwd<T, VEC, 4>(a, st);
  const long long cap = 1LL << 30;
  return launch_k(ln_fwd_long_kernel<T, VEC>, dim3((unsigned)(a.rows < cap ? a.rows : cap)),
                  dim3(1024), 0, st, true, a);
}

// Values a thread of the backward keeps (the sums of its columns stay in
// registers for the whole call); wider rows take the two-pass form.
template <typename T, int VEC, int NV>
cudaError_t bwd(const LnArgs &a, const LnBwdPlan &pl, float *part, cudaStream_t st) {
  return launch_k(ln_bwd_kernel<T, VEC, NV>, dim3(pl.groups), dim3(pl.threads), 0, st, true, a,
                  part);
}

template <typename T, int VEC>
cudaError_t bwd_any(const LnArgs &a, const LnBwdPlan &pl, const float *stat, float *part,
                    cudaStream_t st) {
  if (pl.two_pass) {
    const int cols = 256 * VEC;
    return launch_k(ln_bwd_cols_kernel<T, VEC>, dim3((a.d + cols - 1) / cols, pl.groups), dim3(256),
                    0, st, true, a, stat, part);
  }
  return pl.nv == 1 ? bwd<T, VEC, 1>(a, pl, part, st) : bwd<T, VEC, 8>(a, pl, part, st);
}

template <typename T, int VEC>
cudaError_t stat_any(const LnArgs &a, float *stat, cudaStream_t st) {
  const long long cap = 1LL << 30;
  return launch_k(ln_bwd_stat_kernel<T, VEC>, dim3((unsigned)(a.rows < cap ? a.rows : cap)),
                  dim3(1024), 0, st, true, a, stat);
}

constexpr int kTwoPassGroups = 64;

}  // namespace

cudaError_t launch_layernorm_rows(const LnArgs &a, int bf16, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const int esz = bf16 ? 2 : 4, vec = 16 / esz;
  const bool v = a.d % vec == 0 && rows_aligned(a.x, a.sx, esz) && rows_aligned(a.out, a.so, esz);
  if (bf16) return v ? fwd_any<__nv_bfloat16, 8>(a, st) : fwd_any<__nv_bfloat16, 1>(a, st);
  return v ? fwd_any<float, 4>(a, st) : fwd_any<float, 1>(a, st);
}

LnBwdPlan layernorm_bwd_plan(const LnArgs &a, int bf16) {
  LnBwdPlan pl;
  const int esz = bf16 ? 2 : 4, vec = 16 / esz;
  pl.vec = a.d % vec == 0 && rows_aligned(a.x, a.sx, esz) && rows_aligned(a.dy, a.sg, esz) &&
           rows_aligned(a.out, a.so, esz);
  const int V = pl.vec ? vec : 1;
  pl.nv = a.d <= 1024 * V ? 1 : 8;
  pl.two_pass = a.d > (pl.vec ? 1024 * V : 8192);
  pl.threads = threads_for(a.d, V * pl.nv, 1024);
  // CTAs (each writes one row of partial sums): 1024 threads an SM.
  long long want = pl.two_pass ? kTwoPassGroups
                               : (long long)sm_count() * (pl.threads >= 1024 ? 1 : 1024 / pl.threads);
  pl.groups = (int)(a.rows < want ? a.rows : want);
  return pl;
}

size_t layernorm_bwd_bytes(long long rows, int d) {
  // CTAs of one warp each, or the two-pass form's groups
  const long long most = std::max((long long)sm_count() * 32, (long long)kTwoPassGroups);
  return ((size_t)(rows < most ? rows : most) * 2 * d + (size_t)rows * 2) * sizeof(float);
}

cudaError_t launch_layernorm_bwd_stat(const LnArgs &a, int bf16, const LnBwdPlan &pl, float *stat,
                                      cudaStream_t st) {
  if (bf16)
    return pl.vec ? stat_any<__nv_bfloat16, 8>(a, stat, st) : stat_any<__nv_bfloat16, 1>(a, stat, st);
  return pl.vec ? stat_any<float, 4>(a, stat, st) : stat_any<float, 1>(a, stat, st);
}

cudaError_t launch_layernorm_bwd(const LnArgs &a, int bf16, const LnBwdPlan &pl, const float *stat,
                                 float *part, cudaStream_t st) {
  if (bf16)
    return pl.vec ? bwd_any<__nv_bfloat16, 8>(a, pl, stat, part, st)
                  : bwd_any<__nv_bfloat16, 1>(a, pl, stat, part, st);
  return pl.vec ? bwd_any<float, 4>(a, pl, stat, part, st) : bwd_any<float, 1>(a, pl, stat, part, st);
}

cudaError_t launch_layernorm_bwd_sum(const float *part, int groups, int d, float *dw, float *db,
                                     cudaStream_t st) {
  return launch_k(ln_bwd_sum_kernel, dim3((d + 31) / 32, 2), dim3(1024), 0, st, true, part, groups,
                  d, dw, db);
}

}  // namespace ret
