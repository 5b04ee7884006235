// Building blocks of the selective scan kernels: step sizes, gates, sums over
// the lanes that share a channel, rows of a state.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "rows.cuh"
#include "tc.cuh"

namespace ret {
namespace scan {

// Decays e^(delta A) are ex2() of delta (A log2 e): flushed to zero below 2^-126,
// which loses at most 2^-126 of the state, and shows only where nothing is added
// to it (x = 0).  Keeping them would take a scale and a product more for each
// exponential, the unit that bounds the scan.
constexpr float kLog2e = 1.4426950408889634f;

// 1 / x by the hardware's approximation (2^-23 of itself).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x); 0 and 1 at the ends (the exponential of a very negative x is
// infinite, and its reciprocal 0).
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// ln(1 + e^x) = max(x, 0) + ln(1 + e), e = e^-|x| in (0, 1], where
// ln(1 + e) = 2 artanh(s) = s f(s^2), s = e / (2 + e) <= 1/3.  f(q) = 2 + 2 q / 3 + .. on
// [0, 1/9] by its Chebyshev interpolation of degree 4 (within 2^-26 of itself).
// A difference quotient of ln(1 + e) would lose the small e of small step sizes.
constexpr float kF0 = 2.f, kF1 = 0.6666632294654846f, kF2 = 0.4002459645271301f, kF3 = 0.27965158224105835f,
                kF4 = 0.28157779574394226f;
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(-kLog2e * fabsf(x));
  const float s = e * rcp(2.f + e), q = s * s;
  float p = fmaf(kF4, q, kF3);
  p = fmaf(p, q, kF2);
  p = fmaf(p, q, kF1);
  p = fmaf(p, q, kF0);
  // (NaN: s and with it the sum is NaN, whatever the maximum drops)
  return fmaf(p, s, fmaxf(x, 0.f));
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The same for pairs of channels, on packed arithmetic.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 w = tc::mul2(both(-kLog2e), x), d = tc::add2(both(1.f), make_float2(ex2(w.x), ex2(w.y)));
  return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 silu2(float2 x) { return tc::mul2(x, sigmoid2(x)); }
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 w = tc::mul2(both(-kLog2e), make_float2(fabsf(x.x), fabsf(x.y))), e = make_float2(ex2(w.x), ex2(w.y));
  const float2 d = tc::add2(both(2.f), e), s = tc::mul2(e, make_float2(rcp(d.x), rcp(d.y))), q = tc::mul2(s, s);
  float2 p = tc::fma2(both(kF4), q, both(kF3));
  p = tc::fma2(p, q, both(kF2));
  p = tc::fma2(p, q, both(kF1));
  p = tc::fma2(p, q, both(kF0));
  // (NaN: s and with it the sum is NaN, whatever the maximum drops)
  return tc::fma2(p, s, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Sums of each of N values over groups of L neighbouring lanes times `kStep`
// (L, N powers of two); the lanes share them out: with lane index i in its
// group, v[j] of the result is the sum of value (i % min(L, N)) * N / min(L, N) + j
// for j < N / min(L, N).  Each step halves the values a lane still has to send.
template <int N, int L, int kStep = 1>
__device__ __forceinline__ void share_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  constexpr int M = L < N ? L : N;
  int n = N;
#pragma unroll
  for (int d = M / 2; d >= 1; d >>= 1) {
    const bool up = (lane & (d * kStep)) != 0;
    n >>= 1;
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
      if (j < n) {
        const float keep = up ? v[n + j] : v[j], send = up ? v[j] : v[n + j];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, send, d * kStep);
      }
  }
#pragma unroll
  for (int d = M; d < L; d <<= 1)
#pragma unroll
    for (int j = 0; j < N / M; ++j) v[j] += __shfl_xor_sync(0xffffffffu, v[j], d * kStep);
}

// Four states s0 .. s0 + 3 of a row of S (the missing ones 0).  kVec: the row
// begins on a 16-byte boundary and S is a multiple of 4.
__device__ __forceinline__ float4 load_states(const float *row, int s0, int S, bool vec) {
  if (vec) return s0 < S ? *reinterpret_cast<const float4 *>(row + s0) : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 v;
  v.x = s0 < S ? row[s0] : 0.f;
  v.y = s0 + 1 < S ? row[s0 + 1] : 0.f;
  v.z = s0 + 2 < S ? row[s0 + 2] : 0.f;
  v.w = s0 + 3 < S ? row[s0 + 3] : 0.f;
  return v;
}

__device__ __forceinline__ void store_states(float *row, int s0, int S, bool vec, float4 v) {
  if (vec) {
    if (s0 < S) *reinterpret_cast<float4 *>(row + s0) = v;
    return;
  }
  if (s0 < S) row[s0] = v.x;
  if (s0 + 1 < S) row[s0 + 1] = v.y;
  if (s0 + 2 < S) row[s0 + 2] = v.z;
  if (s0 + 3 < S) row[s0 + 3] = v.w;
}

// Tokens of sequence b: its length within [0, N].
__device__ __forceinline__ int tokens_of(const ScanArgs &a, int b) {
  if (!a.lengths) return a.N;
  const long long n = a.len64 ? reinterpret_cast<const long long *>(a.lengths)[b]
                              : (long long)reinterpret_cast<const int *>(a.lengths)[b];
  return (int)(n < 0 ? 0 : n > a.N ? a.N : n);
}

constexpr int kScan = 128, kLoad = 256, kThreads = kScan + kLoad;

// Channels of a CTA (grid.x counts the blocks of all groups) and tokens at a
// time.  The tile's step sizes take the most shared memory: channels x tokens.
template <int L>
struct Block {
  static constexpr int kChannels = kScan / L;
  static constexpr int kTile = L <= 4 ? 8 * L : 32;
  static constexpr int SP = 4 * L;
  static __host__ __device__ int per_group(int E, int G) { return (E / G + kChannels - 1) / kChannels; }
};

// Two neighbouring channels of a row.
template <typename T>
struct __align__(2 * sizeof(T)) Two {
  T a, b;
};
// To a row; kPair: it begins on the pair's boundary.  n: channels that are there.
template <typename T, bool kPair>
__device__ __forceinline__ void store_two(T *p, int n, float a, float b) {
  if (kPair) {
    if (n > 0) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
      else
        *reinterpret_cast<float2 *>(p) = make_float2(a, b);
    }
  } else {
    if (n > 0) p[0] = from_float<T>(a);
    if (n > 1) p[1] = from_float<T>(b);
  }
}


template <typename T>
__device__ __forceinline__ float2 to_float2(const Two<T> &v) { return make_float2(to_float(v.a), to_float(v.b)); }

template <typename T>
__device__ __forceinline__ void store_pair(T *p, bool pair, int n, float a, float b) {
  if (pair)
    store_two<T, true>(p, n, a, b);
  else
    store_two<T, false>(p, n, a, b);
}

// Four neighbouring channels of a row as they were read; kVec: the row begins on
// the four's boundary.  n: channels that are there.
template <typename T>
struct __align__(4 * sizeof(T)) Four {
  T v[4];
};
template <typename T, bool kVec>
__device__ __forceinline__ Four<T> load_four(const T *p, int n) {
  Four<T> f;
  if (kVec) {
    if constexpr (sizeof(T) == 2) {
      const uint2 w = n > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
      f = *reinterpret_cast<const Four<T> *>(&w);
    } else {
      const float4 w = n > 0 ? *reinterpret_cast<const float4 *>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
      f = *reinterpret_cast<const Four<T> *>(&w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = i < n ? p[i] : from_float<T>(0.f);
  }
  return f;
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_four(T *p, int n, const float (&f)[4]) {
  if (kVec) {
    if (n > 0) {
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
      } else {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_float<T>(f[i]);
  }
}

// Lanes a channel: four states a lane.
inline int lanes_of(int S) {
  int L = 1;
  while (4 * L < S) L *= 2;
  return L;
}

template <typename F>
cudaError_t by_lanes(int S, F f) {
  switch (lanes_of(S)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return f(std::integral_constant<int, 16>());
  }
}

// Does every row of a tensor (and, with E / G a multiple of it, every block of
// channels) begin on a boundary of `step` channels?
inline bool rows_on(const ScanArgs &a, const void *p, const long long s[2], int step, int esz) {
  return !p || (reinterpret_cast<uintptr_t>(p) % (step * esz) == 0 && (a.N <= 1 || s[1] % step == 0) &&
                (a.B <= 1 || s[0] % step == 0));
}

}  // namespace scan
}  // namespace ret
