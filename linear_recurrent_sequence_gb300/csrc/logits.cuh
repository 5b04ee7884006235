// One row of logits walked by a CTA: 16-byte vectors from the row's first
// 16-byte boundary, the few values before and after them one by one, and the
// running maximum and sum of a softmax.
#pragma once

#include "rows.cuh"
#include "tc.cuh"

namespace ret {

// A row of V values: `head` values up to the first 16-byte boundary, `nvec`
// vectors, `tail` values.  Thread t of a CTA of kThreads has the vectors
// t, t + kThreads, ... and, where t < head or t < tail, value t of those.
template <typename T>
struct LogitRow {
  static constexpr int kVec = 16 / (int)sizeof(T);
  const T *p;
  int V, head, nvec, tail;
  __device__ __forceinline__ LogitRow(const T *row, int n) : p(row), V(n) {
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u) / (unsigned)sizeof(T);
    head = off ? min(kVec - (int)off, n) : 0;
    nvec = (n - head) / kVec;
    tail = n - head - nvec * kVec;
  }
  __device__ __forceinline__ int index(int vec) const { return head + vec * kVec; }
  __device__ __forceinline__ int tail_index() const { return head + nvec * kVec; }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Vectors of logits.  max_of: the largest value, NaN if there is one.
template <typename T>
struct LogitVec;

template <>
struct LogitVec<__nv_bfloat16> : Elems<__nv_bfloat16, 8> {
  __device__ __forceinline__ void fill_masked() { raw = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ void mask(int j) {
    uint32_t *w = &raw.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i == j >> 1) w[i] = (j & 1) ? ((w[i] & 0xffffu) | 0xff800000u) : ((w[i] & 0xffff0000u) | 0xff80u);
  }
  template <int N>
  static __device__ __forceinline__ float max_of(const LogitVec (&v)[N]) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&v[0].raw.x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {v[i].raw.x, v[i].raw.y, v[i].raw.z, v[i].raw.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
    }
    return max_nan(__low2float(m), __high2float(m));
  }
};

template <>
struct LogitVec<float> : Elems<float, 4> {
  __device__ __forceinline__ void fill_masked() { raw = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void mask(int j) {
    if (j == 0) raw.x = -INFINITY;
    if (j == 1) raw.y = -INFINITY;
    if (j == 2) raw.z = -INFINITY;
    if (j == 3) raw.w = -INFINITY;
  }
  template <int N>
  static __device__ __forceinline__ float max_of(const LogitVec (&v)[N]) {
    float m = v[0].raw.x;
#pragma unroll
    for (int i = 0; i < N; ++i)
      m = max_nan(max_nan(m, v[i].raw.x), max_nan(max_nan(v[i].raw.y, v[i].raw.z), v[i].raw.w));
    return m;
  }
};

__device__ __forceinline__ float logit_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float logit_of(float x) { return x; }

// Running softmax of the values seen: m the largest, s = sum 2^y and
// u = sum y 2^y with y = (x - m) log2(e) / T.  The exponent is the scaled
// difference, so that neither a mask of the type's lowest value nor a large
// level overflows; below -1000 it is cut (2^y is 0 there, and y 2^y must not
// become infinity times zero).  A NaN or +infinity sets bad: its row has no
// distribution.
struct Softmax {
  float m, s, u;
  bool bad;

  static __device__ __forceinline__ Softmax none() { return {-INFINITY, 0.f, 0.f, false}; }

  // Raises the maximum to at least x.
  __device__ __forceinline__ void raise(float x, float scale) {
    if (!(x <= 3.402823466e38f)) {
      bad = true;
    } else if (x > m) {
      if (m > -INFINITY) {
        const float dy = fmaxf((m - x) * scale, -1000.f), f = ex2(dy);
        u = fmaf(dy, s, u) * f;
        s *= f;
      }
      m = x;
    }
  }
  __device__ __forceinline__ void add(const Softmax &o, float scale) {
    bad |= o.bad;
    Softmax b = o;
    if (b.m > m) {
      raise(b.m, scale);
    } else {
      b.raise(m, scale);
    }
    s += b.s;
    u += b.u;
  }
  // x: at most m.
  __device__ __forceinline__ void take(float x, float scale) {
    const float y = fmaxf((x - (m > -INFINITY ? m : 0.f)) * scale, -1000.f), e = ex2(y);
    s += e;
    u = fmaf(y, e, u);
  }
  template <typename T, int N, bool kEntropy>
  __device__ __forceinline__ void group(const LogitVec<T> (&v)[N], float scale) {
    raise(LogitVec<T>::max_of(v), scale);
    const float mm = m > -INFINITY ? -m : 0.f;
    constexpr int kVec = 16 / (int)sizeof(T);
    float2 s2 = make_float2(0.f, 0.f), u2 = make_float2(0.f, 0.f);
    const float2 mm2 = make_float2(mm, mm), sc2 = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[kVec];
      v[i].get(f);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) {
        float2 y = tc::mul2(tc::add2(make_float2(f[j], f[j + 1]), mm2), sc2);
        if (kEntropy) y = make_float2(fmaxf(y.x, -1000.f), fmaxf(y.y, -1000.f));
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        s2 = tc::add2(s2, e);
        if (kEntropy) u2 = tc::fma2(y, e, u2);
      }
    }
    s += s2.x + s2.y;
    if (kEntropy) u += u2.x + u2.y;
  }
  __device__ __forceinline__ void add_lanes(float scale) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) {
      Softmax o;
      o.m = __shfl_xor_sync(0xffffffffu, m, k);
      o.s = __shfl_xor_sync(0xffffffffu, s, k);
      o.u = __shfl_xor_sync(0xffffffffu, u, k);
      o.bad = __shfl_xor_sync(0xffffffffu, (int)bad, k) != 0;
      add(o, scale);
    }
  }
};

// Joins the CTA's threads' sums (buf: one entry per warp); the result is the
// same in every thread.  Joining two lanes gives both the same bits (the
// operands only change sides).
__device__ __forceinline__ Softmax join_cta(Softmax a, float scale, Softmax *buf) {
  a.add_lanes(scale);
  const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = a;
  __syncthreads();
  Softmax b = lane < nw ? buf[lane] : Softmax::none();
  b.add_lanes(scale);
  return b;
}

}  // namespace ret
