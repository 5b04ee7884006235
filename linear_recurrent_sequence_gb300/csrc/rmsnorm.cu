// Root-mean-square norm over rows of d values, with the residual's addition
// before it, an 8-bit output with scales, and its gradients:
//   h = x + r (rounded to the rows' type, and what is kept is normalised),
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w;
//   with n = h rstd and g = dy w:   dh_total = rstd (g - n mean(g n)) + dh,   dw = sum_rows dy n.
// fp32 arithmetic for bf16 and fp32 rows.  Bound by memory: up to four row
// elements move per value.
#include <algorithm>

#include <cuda_fp8.h>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

constexpr float kE4m3Max = 448.f;

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Sum (or maximum) over the tpr threads of a row: a power of two up to 32
// lanes, or all of the CTA's threads (several warps), through red.
template <bool kMax>
__device__ __forceinline__ float row_join(float x, float *red, int tpr) {
  auto join = [](float p, float q) { return kMax ? max_nan(p, q) : p + q; };
  for (int s = min(tpr, 32) >> 1; s > 0; s >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, s));
  if (tpr <= 32) return x;
  const int lane = threadIdx.x & 31, nw = tpr >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < nw ? red[lane] : 0.f;  // (maxima here are never negative)
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, s));
  return x;
}

template <int V>
__device__ __forceinline__ void load_gain(const float *w, int c, float (&f)[V]) {
  if (!w) {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 1.f;
  } else if constexpr (V == 1) {
    f[0] = w[c];
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(w + c + j);
      f[j] = v.x; f[j + 1] = v.y; f[j + 2] = v.z; f[j + 3] = v.w;
    }
  }
}

// V e4m3 values (rounded to nearest, beyond +-448 that).
template <int V>
struct E4m3 {
  uint32_t w[(V + 3) / 4];
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (V == 1) {
      w[0] = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[j], f[j + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[j + 2], f[j + 3]), __NV_SATFINITE, __NV_E4M3);
        w[j / 4] = lo | hi << 16;
      }
    }
  }
  __device__ __forceinline__ bool operator!=(const E4m3 &o) const {
    uint32_t d = 0;
#pragma unroll
    for (int j = 0; j < (V + 3) / 4; ++j) d |= w[j] ^ o.w[j];
    return d != 0;
  }
  __device__ __forceinline__ void store(uint8_t *p) const {
    if constexpr (V == 1)
      *p = (uint8_t)w[0];
    else if constexpr (V == 4)
      *reinterpret_cast<uint32_t *>(p) = w[0];
    else
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  }
};

// A group's scale from its largest magnitude (of a group of zeros 0), and the
// factor that its values come by: 1 / scale, 1 for zeros, and -1 where the values
// have to be divided, since a subnormal scale's reciprocal may be infinite.
__device__ __forceinline__ float scale_of(float top) { return top / kE4m3Max; }
__device__ __forceinline__ float factor_of(float scale) {
  return scale == 0.f ? 1.f : scale < 1.17549435e-38f ? -1.f : 1.f / scale;
}

template <int V>
__device__ __forceinline__ void times(const float (&f)[V], float k, float (&g)[V]) {
  if constexpr (V == 1) {
    g[0] = f[0] * k;
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 p = tc::mul2(make_float2(f[j], f[j + 1]), make_float2(k, k));
      g[j] = p.x;
      g[j + 1] = p.y;
    }
  }
}

// f / scale, rounded as fp32 divides, as e4m3 values.  The quotient lies between f
// times the factor's neighbours 2^-22 of it on either side (the factor, the
// products and the quotient are each off by at most 2^-24), and so does its e4m3
// value: where the two agree that is it, else (about one value in 200000) it is
// divided for.  16000 x 4096 bf16 124 us; dividing always took 158 where this took
// 128 and a product with the rounded reciprocal, which takes some values across a
// border, 124.
template <int V>
__device__ __forceinline__ void store_scaled(uint8_t *p, float (&f)[V], float factor, const float *scale) {
  E4m3<V> e, o;
  float g[V];
  times<V>(f, factor * (1.f - 0x1p-22f), g);
  e.set(g);
  times<V>(f, factor * (1.f + 0x1p-22f), g);
  o.set(g);
  if (e != o || factor < 0.f) {
    const float s = *scale;
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] /= s;
    e.set(f);
  }
  e.store(p);
}

// The group of column c.
__device__ __forceinline__ int group_of(const RmsArgs &a, int c) {
  return a.groups == 1 ? 0 : a.shift >= 0 ? c >> a.shift : c / a.group;
}

// Rounds to the rows' type, as what is kept of the sum is.
template <typename T, int V>
__device__ __forceinline__ void add_rounded(const Elems<T, V> &a, const Elems<T, V> &b, Elems<T, V> &h) {
  float f[V], g[V];
  a.get(f);
  b.get(g);
#pragma unroll
  for (int j = 0; j < V; ++j) f[j] += g[j];
  h.set(f);
}

// The vectors of one row that a thread reads, on their way.
template <typename T, int V, int NV>
struct RowIn {
  Elems<T, V> v[NV];
  __device__ __forceinline__ void load(const T *p, int tpr, int t, int d) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + t) * V;
      if (c < d) v[i].load(p + c);
    }
  }
};

// tpr threads a row, NV vectors of V values a thread, interleaved; the row
// stays in registers, and the next one is on its way meanwhile.  kQuant: e4m3
// output.  16384 x 4096 bf16 with a residual 86 us (6.2 TB/s), without the next
// row's loads 105; e4m3 with groups of 128 16000 x 4096 124 us (3.7 TB/s: two more
// meetings of the CTA a row; barriers, shuffles and shared atomics).  fp32 rows above
// 8192 spill 48 bytes, 396 with e4m3 (1500 x 16384 138 us).
template <typename T, int V, int NV, bool kQuant>
__global__ void __launch_bounds__(512)
rms_fwd_kernel(const RmsArgs a, int tpr) {
  extern __shared__ unsigned amax[];  // [rows of the CTA][groups]
  __shared__ float red[2][32];
  pdl_wait();
  const int row_in = threadIdx.x / tpr, t = threadIdx.x - row_in * tpr, per = blockDim.x / tpr;
  const float inv_d = 1.f / (float)a.d;
  RowIn<T, V, NV> xn, rn;
  auto ahead = [&](long long r) {
    if (r >= a.rows) return;
    xn.load(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), tpr, t, a.d);
    if (a.r) rn.load(reinterpret_cast<const T *>(a.r) + row_offset(a.sr, r), tpr, t, a.d);
  };
  ahead((long long)blockIdx.x * per + row_in);
  int par = 0;
  for (long long r0 = (long long)blockIdx.x * per; r0 < a.rows; r0 += (long long)gridDim.x * per, par ^= 1) {
    const long long r = r0 + row_in;
    const bool live = r < a.rows;
    Elems<T, V> h[NV];
    float s = 0.f;
    if (kQuant) {
      for (int i = threadIdx.x; i < per * a.groups; i += blockDim.x) amax[i] = 0u;
    }
    if (live) {
      T *ho = a.r ? reinterpret_cast<T *>(a.h) + row_offset(a.sh, r) : nullptr;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * V;
        if (c < a.d) {
          if (a.r) {
            add_rounded<T, V>(xn.v[i], rn.v[i], h[i]);
            h[i].store(ho + c);
          } else {
            h[i] = xn.v[i];
          }
          float f[V];
          h[i].get(f);
#pragma unroll
          for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
        }
      }
    }
    ahead(r + (long long)gridDim.x * per);
    s = row_join<false>(s, red[par], tpr);
    const float rstd = rsqrtf(fmaf(s, inv_d, a.eps));
    if (live && t == 0 && a.rstd) a.rstd[r] = rstd;
    if (!kQuant) {
      if (live) {
        T *y = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * tpr + t) * V;
          if (c < a.d) {
            float f[V], w[V];
            h[i].get(f);
            load_gain<V>(a.w, c, w);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = f[j] * rstd * w[j];
            h[i].set(f);
            h[i].store(y + c);
          }
        }
      }
    } else {
      if (tpr <= 32) __syncthreads();  // the maxima are cleared (wider rows met in the sum)
      unsigned *top = amax + row_in * a.groups;
      float f[NV][V], row_top = 0.f;
      const bool warps = tpr >= 32 && a.group % (32 * V) == 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * V;
        float m = 0.f;
        if (live && c < a.d) {
          float w[V];
          h[i].get(f[i]);
          load_gain<V>(a.w, c, w);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            f[i][j] = f[i][j] * rstd * w[j];
            m = max_nan(m, fabsf(f[i][j]));
          }
        }
        // A warp whose vectors (neighbours) are of one group joins them first, or all
        // of a thread's vectors do; then one atomic each (a maximum does not depend
        // on the order of its atomics; as bits NaN is above all numbers).  Half a
        // warp's vectors joined by shuffles: 16000 x 4096 bf16 with groups of 128
        // 128 us for 124, 512 x 4096 13 for both.
        if (a.groups == 1) {
          row_top = max_nan(row_top, m);
        } else if (warps) {
          const unsigned top32 = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
          if ((threadIdx.x & 31) == 0 && live && c < a.d) atomicMax(top + group_of(a, c), top32);
        } else if (live && c < a.d) {
          atomicMax(top + group_of(a, c), __float_as_uint(m));
        }
      }
      if (a.groups == 1) {
        if (tpr >= 32) row_top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(row_top)));
        if (live && (tpr < 32 || (threadIdx.x & 31) == 0)) atomicMax(top, __float_as_uint(row_top));
      }
      __syncthreads();
      for (int i = threadIdx.x; i < per * a.groups; i += blockDim.x) {
        const float scale = scale_of(__uint_as_float(amax[i]));
        if (r0 + i / a.groups < a.rows) a.scales[r0 * a.groups + i] = scale;
        amax[i] = __float_as_uint(factor_of(scale));
      }
      __syncthreads();
      if (live) {
        uint8_t *y = reinterpret_cast<uint8_t *>(a.out) + row_offset(a.so, r);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * tpr + t) * V;
          if (c < a.d) {
            const int g = group_of(a, c);
            store_scaled<V>(y + c, f[i], __uint_as_float(top[g]), a.scales + r * a.groups + g);
          }
        }
      }
      __syncthreads();  // the maxima are free again
    }
  }
  pdl_launch_dependents();
}

// Rows too long for registers: read again for the output (the kept sum, or x).
template <typename T, int V, bool kQuant>
__global__ void __launch_bounds__(1024)
rms_fwd_long_kernel(const RmsArgs a) {
  __shared__ float red[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int step = blockDim.x * V, first = threadIdx.x * V;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    const T *q = a.r ? reinterpret_cast<const T *>(a.r) + row_offset(a.sr, r) : nullptr;
    T *ho = a.r ? reinterpret_cast<T *>(a.h) + row_offset(a.sh, r) : nullptr;
    float s = 0.f, f[V], w[V];
    Elems<T, V> e, o;
    for (int c = first; c < a.d; c += step) {
      e.load(x + c);
      if (q) {
        o.load(q + c);
        add_rounded<T, V>(e, o, e);
        e.store(ho + c);
      }
      e.get(f);
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
    }
    s = row_join<false>(s, red[0], blockDim.x);
    const float rstd = rsqrtf(s / (float)a.d + a.eps);
    if (threadIdx.x == 0 && a.rstd) a.rstd[r] = rstd;
    const T *from = q ? ho : x;  // (each thread reads what it wrote itself)
    if (!kQuant) {
      T *y = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
      for (int c = first; c < a.d; c += step) {
        e.load(from + c);
        e.get(f);
        load_gain<V>(a.w, c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = f[j] * rstd * w[j];
        e.set(f);
        e.store(y + c);
      }
    } else {
      uint8_t *y = reinterpret_cast<uint8_t *>(a.out) + row_offset(a.so, r);
      // a warp for each group, or all of them for wide ones (what others kept of
      // the sum is visible: several warps met above, the lanes of one meet here,
      // since its shuffles do not order memory)
      __syncwarp();
      const bool wide = a.group > 1024;
      const int lead = (wide ? threadIdx.x : threadIdx.x & 31) * V, hop = (wide ? blockDim.x : 32) * V;
      for (int g = wide ? 0 : threadIdx.x >> 5; g < a.groups; g += wide ? 1 : blockDim.x >> 5) {
        const int c1 = min(a.d, (g + 1) * a.group);
        float m = 0.f;
        for (int c = g * a.group + lead; c < c1; c += hop) {
          e.load(from + c);
          e.get(f);
          load_gain<V>(a.w, c, w);
#pragma unroll
          for (int j = 0; j < V; ++j) m = max_nan(m, fabsf(f[j] * rstd * w[j]));
        }
        m = row_join<true>(m, red[1], wide ? blockDim.x : 32);
        const float scale = scale_of(m), factor = factor_of(scale);
        if (lead == 0) a.scales[r * a.groups + g] = scale;
        for (int c = g * a.group + lead; c < c1; c += hop) {
          e.load(from + c);
          e.get(f);
          load_gain<V>(a.w, c, w);
#pragma unroll
          for (int j = 0; j < V; ++j) f[j] = f[j] * rstd * w[j];
          store_scaled<V>(y + c, f, factor, &scale);
        }
        if (wide) __syncthreads();  // red is free again
      }
    }
    __syncthreads();
  }
}

// dx of the rows of the CTA, and its sums of dy n: a thread keeps those of its
// own columns in registers.  8192 x 4096 bf16 64 us (4.2 TB/s; a row's steps, the
// shuffles of its sum first, at the two CTAs an SM that 114 registers leave; half
// the issue slots), without the next row's loads 75; 60000 x 1001 value by value 253.
// fp32 113 us; four vectors of it a thread spill 80 bytes.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512)
rms_bwd_kernel(const RmsArgs a, int tpr, float *__restrict__ part) {
  extern __shared__ float sums[];  // [rows of the CTA][d] where there are several
  __shared__ float red[2][32];
  pdl_wait();
  const int row_in = threadIdx.x / tpr, t = threadIdx.x - row_in * tpr, per = blockDim.x / tpr;
  const float inv_d = 1.f / (float)a.d;
  float dw[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
  int par = 0;
  constexpr bool kAhead = V == 1 ? NV <= 8 : NV * V <= 16;  // (else the registers hold one row)
  RowIn<T, V, NV> hn, gn, pn;
  float rn = 0.f;
  auto ahead = [&](long long r) {
    if (r >= a.rows) return;
    hn.load(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), tpr, t, a.d);
    gn.load(reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r), tpr, t, a.d);
    if (a.dh) pn.load(reinterpret_cast<const T *>(a.dh) + row_offset(a.sdh, r), tpr, t, a.d);
    rn = a.rstd[r];
  };
  if (kAhead) ahead((long long)blockIdx.x * per + row_in);
  for (long long r0 = (long long)blockIdx.x * per; r0 < a.rows; r0 += (long long)gridDim.x * per, par ^= 1) {
    const long long r = r0 + row_in;
    const bool live = r < a.rows;
    Elems<T, V> h[NV], g[NV], p[NV];
    float s = 0.f;
    if (!kAhead) ahead(r);
    const float rstd = rn;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      h[i] = hn.v[i];
      g[i] = gn.v[i];
      p[i] = pn.v[i];
    }
    if (kAhead) ahead(r + (long long)gridDim.x * per);
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * V;
        if (c < a.d) {
          float f[V], q[V], w[V];
          h[i].get(f);
          g[i].get(q);
          load_gain<V>(a.w, c, w);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float n = f[j] * rstd;
            dw[i][j] = fmaf(q[j], n, dw[i][j]);
            s = fmaf(q[j] * w[j], n, s);
          }
        }
      }
    }
    s = row_join<false>(s, red[par], tpr);
    const float k = -s * inv_d;
    if (live) {
      T *dx = reinterpret_cast<T *>(a.out) + row_offset(a.so, r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + t) * V;
        if (c < a.d) {
          float f[V], q[V], w[V], o[V];
          h[i].get(f);
          g[i].get(q);
          load_gain<V>(a.w, c, w);
          if (a.dh) p[i].get(o);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float v = fmaf(f[j] * rstd, k, q[j] * w[j]);
            o[j] = a.dh ? fmaf(v, rstd, o[j]) : v * rstd;
          }
          h[i].set(o);
          h[i].store(dx + c);
        }
      }
    }
  }
  pdl_launch_dependents();
  if (!part) return;
  float *out = part + (size_t)blockIdx.x * a.d;
  float *mine = per > 1 ? sums + (size_t)row_in * a.d : out;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + t) * V;
    if (c < a.d)
#pragma unroll
      for (int j = 0; j < V; ++j) mine[c + j] = dw[i][j];
  }
  if (per == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    float v = sums[c];
    for (int i = 1; i < per; ++i) v += sums[(size_t)i * a.d + c];
    out[c] = v;
  }
}

// Rows too long for registers, in two passes: mean(g n) of each row, then dx
// and the column sums by blocks of columns.
template <typename T, int V>
__global__ void __launch_bounds__(1024)
rms_bwd_stat_kernel(const RmsArgs a, float *__restrict__ stat) {
  __shared__ float red[32];
  pdl_launch_dependents();
  pdl_wait();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T *x = reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r);
    const T *dy = reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r);
    const float rstd = a.rstd[r];
    float s = 0.f;
    for (int c = threadIdx.x * V; c < a.d; c += blockDim.x * V) {
      Elems<T, V> h, g;
      h.load(x + c);
      g.load(dy + c);
      float f[V], q[V], w[V];
      h.get(f);
      g.get(q);
      load_gain<V>(a.w, c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(q[j] * w[j], f[j] * rstd, s);
    }
    s = row_join<false>(s, red, blockDim.x);
    if (threadIdx.x == 0) stat[r] = s / (float)a.d;
    __syncthreads();
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256)
rms_bwd_cols_kernel(const RmsArgs a, const float *__restrict__ stat, float *__restrict__ part) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (c >= a.d) return;
  float dw[V], w[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = 0.f;
  load_gain<V>(a.w, c, w);
  for (long long r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float rstd = a.rstd[r], k = -stat[r];
    Elems<T, V> h, g, p;
    h.load(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r) + c);
    g.load(reinterpret_cast<const T *>(a.dy) + row_offset(a.sg, r) + c);
    if (a.dh) p.load(reinterpret_cast<const T *>(a.dh) + row_offset(a.sdh, r) + c);
    float f[V], q[V], o[V];
    h.get(f);
    g.get(q);
    if (a.dh) p.get(o);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float n = f[j] * rstd, v = fmaf(n, k, q[j] * w[j]);
      dw[j] = fmaf(q[j], n, dw[j]);
      o[j] = a.dh ? fmaf(v, rstd, o[j]) : v * rstd;
    }
    h.set(o);
    h.store(reinterpret_cast<T *>(a.out) + row_offset(a.so, r) + c);
  }
  if (!part) return;
#pragma unroll
  for (int j = 0; j < V; ++j) part[(size_t)blockIdx.y * a.d + c + j] = dw[j];
}

// 16-byte vectors need every row of every operand on a 16-byte boundary.
bool rows_on(const void *p, const RowSet &s, int esz, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (s.n1 == 1 || s.s1 * esz % bytes == 0) &&
         (s.n0 == 1 || s.s0 * esz % bytes == 0);
}

// Threads a row for n vectors, NV a thread: lanes of a warp (a power of two) or whole warps.
int threads_per_row(int n, int most) {
  const int t = (n + most - 1) / most;
  if (t > 16) return (t + 31) / 32 * 32;
  int p = 1;
  while (p < t) p *= 2;
  return p;
}

template <typename T, int V, bool kQuant>
cudaError_t fwd_any(const RmsArgs &a, cudaStream_t st) {
  const int n = (a.d + V - 1) / V, sms = device_sms();
  // At most 512 threads a row: 8 values a thread for few rows (all of them at
  // once), else 16 (more bytes in flight beside the next row's), or 32.
  auto go = [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    const int tpr = threads_per_row(n, NV), threads = tpr > 32 ? tpr : 128, per = threads / tpr;
    const long long want = (a.rows + per - 1) / per, most = (long long)sms * std::max(1, 1024 / threads);
    const size_t smem = kQuant ? (size_t)per * a.groups * 4 : 0;
    return launch_k(rms_fwd_kernel<T, V, NV, kQuant>, dim3((unsigned)std::min(want, most)), dim3(threads), smem, st, true, a, tpr);
  };
  // A CTA a row, 16 values a thread (long rows: 1024 threads), read again for the
  // output.  (8 a thread: 16000 x 4099 bf16 with e4m3 output 338 us for 262, now 267.)
  auto again = [&] {
    const long long cap = 1LL << 30;
    const int threads = a.d > 512 * 16 ? 1024 : ((a.d + 15) / 16 + 31) / 32 * 32;
    return launch_k(rms_fwd_long_kernel<T, V, kQuant>, dim3((unsigned)std::min(a.rows, cap)), dim3(threads), 0, st, true, a);
  };
  const bool few = a.rows * ((a.d + 7) / 8) <= (long long)sms * 1024;
  if (a.d <= 512 * 8 && (few || a.d <= 256)) return go(std::integral_constant<int, 8 / V>());
  // Value by value the registers of a long row spill: 16000 x 4099 bf16 with e4m3
  // output 1011 us (read again 262), 5000 x 12001 without 773 (219).
  if constexpr (V == 1) {
    if constexpr (!kQuant)
      if (a.d <= 512 * 16) return go(std::integral_constant<int, 16>());
    return again();
  } else {
    if (a.d <= 512 * 16) return go(std::integral_constant<int, 16 / V>());
    if (a.d <= 512 * 32) return go(std::integral_constant<int, 32 / V>());
    return again();
  }
}

template <bool kQuant>
cudaError_t launch_fwd(RmsArgs a, int bf16, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  a.shift = -1;
  for (int i = 3; i < 30; ++i)
    if (a.group == 1 << i) a.shift = i;
  const int esz = bf16 ? 2 : 4, vec = 16 / esz;
  const bool v = a.d % vec == 0 && rows_on(a.x, a.sx, esz, 16) && (!a.r || (rows_on(a.r, a.sr, esz, 16) && rows_on(a.h, a.sh, esz, 16))) &&
                 rows_on(a.out, a.so, kQuant ? 1 : esz, kQuant ? vec : 16) && reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
  if (bf16) return v ? fwd_any<__nv_bfloat16, 8, kQuant>(a, st) : fwd_any<__nv_bfloat16, 1, kQuant>(a, st);
  return v ? fwd_any<float, 4, kQuant>(a, st) : fwd_any<float, 1, kQuant>(a, st);
}

constexpr int kTwoPassGroups = 64;

template <typename T, int V>
cudaError_t bwd_any(const RmsArgs &a, const RmsBwdPlan &pl, const float *stat, float *part, cudaStream_t st) {
  if (pl.two_pass) {
    const int cols = 256 * V;
    return launch_k(rms_bwd_cols_kernel<T, V>, dim3((a.d + cols - 1) / cols, pl.groups), dim3(256), 0, st, true, a, stat, part);
  }
  const int threads = pl.tpr > 32 ? pl.tpr : 128, per = threads / pl.tpr;
  const size_t smem = per > 1 ? (size_t)per * a.d * sizeof(float) : 0;
  if constexpr (V == 8)
    if (pl.values == 32)
      return launch_k(rms_bwd_kernel<T, V, 32 / V>, dim3(pl.groups), dim3(threads), smem, st, true, a, pl.tpr, part);
  if (pl.values == 16)
    return launch_k(rms_bwd_kernel<T, V, 16 / V>, dim3(pl.groups), dim3(threads), smem, st, true, a, pl.tpr, part);
  return launch_k(rms_bwd_kernel<T, V, 8 / V>, dim3(pl.groups), dim3(threads), smem, st, true, a, pl.tpr, part);
}

template <typename T, int V>
cudaError_t stat_any(const RmsArgs &a, float *stat, cudaStream_t st) {
  const long long cap = 1LL << 30;
  return launch_k(rms_bwd_stat_kernel<T, V>, dim3((unsigned)std::min(a.rows, cap)), dim3(1024), 0, st, true, a, stat);
}

}  // namespace

cudaError_t launch_rmsnorm_fwd(const RmsArgs &a, int bf16, cudaStream_t st) { return launch_fwd<false>(a, bf16, st); }
cudaError_t launch_rmsnorm_quant(const RmsArgs &a, int bf16, cudaStream_t st) { return launch_fwd<true>(a, bf16, st); }

// V: values of a vector.
static RmsBwdPlan plan_of(long long rows, int d, int V) {
  RmsBwdPlan pl;
  pl.vec = V > 1;
  const int n = (d + V - 1) / V;
  // At most 512 threads a row with 8 or 16 values each, for 16-byte vectors of
  // bf16 (whose rows take half the registers) 32.
  pl.values = d <= 256 ? 8 : d <= 512 * 16 ? 16 : 32;
  if (d > 512 * (V == 8 ? 32 : 16)) {
    pl.two_pass = true;
    pl.groups = (int)std::min<long long>(rows, kTwoPassGroups);
    return pl;
  }
  pl.tpr = threads_per_row(n, pl.values / V);
  const int threads = pl.tpr > 32 ? pl.tpr : 128, per = threads / pl.tpr;
  const long long want = (rows + per - 1) / per, most = (long long)device_sms() * std::min(16, std::max(1, 1024 / threads));
  pl.groups = (int)std::min(want, most);
  return pl;
}

RmsBwdPlan rmsnorm_bwd_plan(const RmsArgs &a, int bf16) {
  const int esz = bf16 ? 2 : 4, vec = 16 / esz;
  const bool v = a.d % vec == 0 && rows_on(a.x, a.sx, esz, 16) && rows_on(a.dy, a.sg, esz, 16) &&
                 (!a.dh || rows_on(a.dh, a.sdh, esz, 16)) && rows_on(a.out, a.so, esz, 16) &&
                 reinterpret_cast<uintptr_t>(a.w) % 16 == 0;
  return plan_of(a.rows, a.d, v ? vec : 1);
}

// Of the plan with vectors or without, whichever takes more.
size_t rmsnorm_bwd_bytes(long long rows, int d, int bf16) {
  size_t most = 0;
  for (const int V : {1, bf16 ? 8 : 4}) {
    const RmsBwdPlan pl = plan_of(rows, d, V);
    most = std::max(most, ((size_t)pl.groups * d + (pl.two_pass ? (size_t)rows : 0)) * sizeof(float));
  }
  return most;
}

cudaError_t launch_rmsnorm_bwd_stat(const RmsArgs &a, int bf16, const RmsBwdPlan &pl, float *stat, cudaStream_t st) {
  if (bf16) return pl.vec ? stat_any<__nv_bfloat16, 8>(a, stat, st) : stat_any<__nv_bfloat16, 1>(a, stat, st);
  return pl.vec ? stat_any<float, 4>(a, stat, st) : stat_any<float, 1>(a, stat, st);
}

cudaError_t launch_rmsnorm_bwd(const RmsArgs &a, int bf16, const RmsBwdPlan &pl, const float *stat, float *part,
                               cudaStream_t st) {
  if (bf16) return pl.vec ? bwd_any<__nv_bfloat16, 8>(a, pl, stat, part, st) : bwd_any<__nv_bfloat16, 1>(a, pl, stat, part, st);
  return pl.vec ? bwd_any<float, 4>(a, pl, stat, part, st) : bwd_any<float, 1>(a, pl, stat, part, st);
}

}  // namespace ret
