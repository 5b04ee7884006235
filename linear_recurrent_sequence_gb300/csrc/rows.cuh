// Row-wise building blocks of the LayerNorm and logits kernels: rows of a
// strided matrix, 16-byte vectors of bf16 or fp32 elements, warp sums.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "tc.cuh"

namespace ret {

// Element offset of row r of an n0 x n1 set of rows.
__device__ __forceinline__ long long row_offset(const RowSet &s, long long r) {
  if (s.n0 == 1) return r * s.s1;
  // (a 64-bit division costs over a hundred instructions)
  const long long i = (r | s.n1) >> 32 ? r / s.n1 : (long long)((uint32_t)r / (uint32_t)s.n1);
  return i * s.s0 + (r - i * s.n1) * s.s1;
}

// 16 bytes of a row that is read once: not kept in L1, which is left to the
// parameters that every row reads.
__device__ __forceinline__ uint4 load_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// VEC consecutive elements of type T as floats.  VEC is 16 / sizeof(T) (the
// address is then 16-byte aligned) or 1.
template <typename T, int VEC>
struct Elems;

template <>
struct Elems<__nv_bfloat16, 8> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = load_stream(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = raw;
  }
};

template <>
struct Elems<float, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const float *p) {
    const uint4 v = load_stream(p);
    raw = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                      __uint_as_float(v.w));
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = raw.x; f[1] = raw.y; f[2] = raw.z; f[3] = raw.w;
  }
  __device__ __forceinline__ void set(const float (&f)[4]) {
    raw = make_float4(f[0], f[1], f[2], f[3]);
  }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = raw; }
};

template <>
struct Elems<__nv_bfloat16, 1> {
  __nv_bfloat16 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { raw = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(raw); }
  __device__ __forceinline__ void set(const float (&f)[1]) { raw = __float2bfloat16_rn(f[0]); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *p = raw; }
};

template <>
struct Elems<float, 1> {
  float raw;
  __device__ __forceinline__ void load(const float *p) { raw = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = raw; }
  __device__ __forceinline__ void set(const float (&f)[1]) { raw = f[0]; }
  __device__ __forceinline__ void store(float *p) const { *p = raw; }
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}

// 2^x, flushed to zero below 2^-126 (the hardware's approximation).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace ret
