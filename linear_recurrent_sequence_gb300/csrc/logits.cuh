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
  __device__ __forceinline__ void floor_at(float x) {
    const __nv_bfloat162 f = __float2bfloat162_rn(x);
    uint32_t *w = &raw.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), f);
      w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
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
  __device__ __forceinline__ void floor_at(float x) {
    raw = make_float4(fmaxf(raw.x, x), fmaxf(raw.y, x), fmaxf(raw.z, x), fmaxf(raw.w, x));
  }
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

__device__ __forceinline__ float redux_max(float x) {  // over the warp; a NaN counts as absent
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fffffff); }
constexpr float kFltMax = 3.402823466e38f;

// Softmax of a set of values: m the largest, s = sum 2^y and u = sum y 2^y
// with y = (x - m) log2(e) / T.  A NaN or +infinity among them sets bad: they
// have no distribution.
struct Softmax {
  float m, s, u;
  int bad;
};

// The temperature's scale log2(e) / T and what follows from it.  Up to `high`
// in size a maximum m has m scale within 2^22, so that the product's rounding,
// which the exponents below carry until all() takes it out, is at most 1/8.
// `low` stands for a logit below it (its 2^y is 0, and y 2^y is not infinity
// times zero as it would be for -infinity).
struct Scale {
  float scale, high, low;
  __device__ __forceinline__ explicit Scale(float sc)
      : scale(sc), high(4194304.f / sc), low(-1e36f / fmaxf(sc, 1.f)) {}
};

// The softmax of the values that a warp's threads walk over.  m is the same in
// all lanes (one reduction of the lanes' maxima for each group of vectors), so
// the sums are moved to a new maximum by a branch that the whole warp takes,
// and seldom; the sums are packed pairs of a lane's own.
// One fused multiply-add gives a pair's exponents: they are relative to the
// rounded product m scale, which all() corrects.  Where the maximum is beyond
// `high` (so far only values of a finite mask, or a low temperature) the
// rounding would be as large as any exponent, and the difference is taken
// first; the exponents are then relative to m itself.
struct WarpSoftmax {
  float m = -INFINITY, own = -INFINITY;  // own: the lane's largest value, NaN if it met one
  float2 s = {0.f, 0.f}, u = {0.f, 0.f};

  template <typename T, int N, bool kEntropy>
  __device__ __forceinline__ void group(const LogitVec<T> (&v)[N], const Scale &c) {
    const float top = LogitVec<T>::max_of(v);
    own = max_nan(own, top);
    raise<kEntropy>(redux_max(top), c);
    constexpr int kVec = 16 / (int)sizeof(T);
    if (fabsf(m) <= c.high) {
      const float2 sc2 = make_float2(c.scale, c.scale), mm2 = make_float2(-__fmul_rn(m, c.scale), -__fmul_rn(m, c.scale));
#pragma unroll
      for (int i = 0; i < N; ++i) {
        LogitVec<T> w = v[i];
        if (kEntropy) w.floor_at(c.low);
        float f[kVec];
        w.get(f);
#pragma unroll
        for (int j = 0; j < kVec; j += 2) take<kEntropy>(tc::fma2(make_float2(f[j], f[j + 1]), sc2, mm2));
      }
    } else if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float f[kVec];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < kVec; j += 2) take_far<kEntropy>(f[j], f[j + 1], c.scale);
      }
    }
  }
  // One value a lane (-infinity: none).
  template <bool kEntropy>
  __device__ __forceinline__ void single(float x, const Scale &c) {
    own = max_nan(own, x);
    raise<kEntropy>(redux_max(x), c);
    if (fabsf(m) <= c.high)
      take<kEntropy>(make_float2(fmaf(fmaxf(x, c.low), c.scale, -__fmul_rn(m, c.scale)), -1000.f));
    else if (m > -INFINITY)
      take_far<kEntropy>(x, -INFINITY, c.scale);
  }
  // The warp's result, in all lanes.
  template <bool kEntropy>
  __device__ __forceinline__ Softmax all(const Scale &c) const {
    Softmax r;
    r.m = m;
    r.s = warp_sum(s.x + s.y);
    r.u = kEntropy ? warp_sum(u.x + u.y) : 0.f;
    if (fabsf(m) <= c.high) {
      const float off = fmaf(m, c.scale, -__fmul_rn(m, c.scale)), f = ex2(-off);
      r.u = __fmul_rn(fmaf(-off, r.s, r.u), f);
      r.s = __fmul_rn(r.s, f);
    }
    r.bad = __any_sync(0xffffffffu, !(own <= kFltMax));
    return r;
  }

 private:
  // The exponent that moves the sums from m to `top`, each as group() refers to it.
  __device__ __forceinline__ float shift(float top, const Scale &c) const {
    const float pm = __fmul_rn(m, c.scale), pt = __fmul_rn(top, c.scale);
    const bool near_m = fabsf(m) <= c.high, near_top = fabsf(top) <= c.high;
    if (near_m) return near_top ? __fsub_rn(pm, pt) : -fmaf(top, c.scale, -pm);
    return near_top ? fmaf(m, c.scale, -pt) : __fmul_rn(__fsub_rn(m, top), c.scale);
  }
  template <bool kEntropy>
  __device__ __forceinline__ void raise(float top, const Scale &c) {
    if (!(top > m)) return;
    if (m > -INFINITY) {
      // (a difference of infinities is one of values far apart: -1000 too)
      const float dy = fmaxf(shift(top, c), -1000.f), f = ex2(dy);
      const float2 f2 = make_float2(f, f);
      if (kEntropy) u = tc::mul2(tc::fma2(make_float2(dy, dy), s, u), f2);
      s = tc::mul2(s, f2);
    }
    m = top;
  }
  template <bool kEntropy>
  __device__ __forceinline__ void take(float2 y) {
    const float2 e = make_float2(ex2(y.x), ex2(y.y));
    s = tc::add2(s, e);
    if (kEntropy) u = tc::fma2(y, e, u);
  }
  template <bool kEntropy>
  __device__ __forceinline__ void take_far(float a, float b, float scale) {
    take<kEntropy>(make_float2(fmaxf((a - m) * scale, -1000.f), fmaxf((b - m) * scale, -1000.f)));
  }
};

// Joins up to kLanes parts (a power of two), one in each of the first kLanes
// lanes and again in every kLanes after them; an absent part has m = -infinity
// and zeros.
template <bool kEntropy, int kLanes>
__device__ __forceinline__ Softmax join_lanes(const Softmax &p, float scale) {
  Softmax r;
  r.m = redux_max(p.m);
  const bool some = p.m > -INFINITY;
  const float dy = some ? fmaxf((p.m - r.m) * scale, -1000.f) : 0.f, f = some ? ex2(dy) : 0.f;
  // (no contraction: the same bits wherever this is inlined)
  r.s = __fmul_rn(p.s, f);
  r.u = kEntropy ? __fmul_rn(fmaf(dy, p.s, p.u), f) : 0.f;
#pragma unroll
  for (int k = kLanes / 2; k > 0; k >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, k);
    if (kEntropy) r.u += __shfl_xor_sync(0xffffffffu, r.u, k);
  }
  r.bad = __any_sync(0xffffffffu, p.bad);
  return r;
}

// ------------------------------------------------------------ clusters
// A row may be shared by the CTAs of a cluster, a slice of vectors each.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Halves of a barrier after which this CTA's shared memory is its own again:
// every CTA arrives when it has read the others', and waits before it writes
// what they read (or ends).  It orders no memory, so it does not wait for
// the stores of results.
__device__ __forceinline__ void cluster_have_read() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_read() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// A 32-bit word of CTA `rank`'s shared memory, at the place of `local` in this one's.
__device__ __forceinline__ uint32_t cluster_word(const void *local, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// Joins the CTA's first kWarps warps, and the cluster's CTAs where
// there are several: the same result in every thread.  parts: shared,
// [kWarps]; mine: shared, one.
// In a cluster the caller then has to arrive and wait (cluster_have_read,
// cluster_wait_read) before `mine` is written again.
template <bool kEntropy, int kWarps>
__device__ __forceinline__ Softmax join_row(const Softmax &warp, float scale, uint32_t ctas,
                                            Softmax *parts, Softmax *mine) {
  const int lane = threadIdx.x & 31;
  if (lane == 0 && threadIdx.x < kWarps * 32) parts[threadIdx.x >> 5] = warp;
  __syncthreads();
  Softmax r = join_lanes<kEntropy, kWarps>(parts[lane & (kWarps - 1)], scale);
  if (ctas == 1) return r;
  if (threadIdx.x == 0) *mine = r;
  cluster_sync();
  Softmax p = {-INFINITY, 0.f, 0.f, 0};
  const uint32_t c = lane & 7;
  if (c < ctas) {
    p.m = __uint_as_float(cluster_word(&mine->m, c));
    p.s = __uint_as_float(cluster_word(&mine->s, c));
    p.u = __uint_as_float(cluster_word(&mine->u, c));
    p.bad = (int)cluster_word(&mine->bad, c);
  }
  return join_lanes<kEntropy, 8>(p, scale);
}

// The vectors of a row that this CTA walks over, and whether it also has the
// values before (first) and after (last) them: lanes 0..7 and 8..15 of warp 0
// have one of those each.
struct RowSlice {
  int v0, v1;
  bool first, last;
  template <typename T>
  __device__ __forceinline__ RowSlice(const LogitRow<T> &row, uint32_t ctas, uint32_t rank) {
    const int each = (row.nvec + (int)ctas - 1) / (int)ctas;
    v0 = min((int)rank * each, row.nvec);
    v1 = min(v0 + each, row.nvec);
    first = rank == 0;
    last = rank + 1 == ctas;
  }
  template <typename T>
  __device__ __forceinline__ bool has(const LogitRow<T> &row, int i) const {
    if (i < row.head) return first;
    if (i >= row.tail_index()) return last;
    const int v = (i - row.head) / LogitRow<T>::kVec;
    return v >= v0 && v < v1;
  }
  // Index of the single value of this thread, -1 if it has none.
  template <typename T>
  __device__ __forceinline__ int single(const LogitRow<T> &row) const {
    const int t = threadIdx.x;
    if (t < 8) return first && t < row.head ? t : -1;
    return t < 16 && last && t - 8 < row.tail ? row.tail_index() + t - 8 : -1;
  }
};

// CTAs a row: as many as bring a slice down to `most` bytes, and more while
// all of them fit the SMs at once (`slots`) and slices stay above 8 KB.
inline int row_ctas(long long rows, long long row_bytes, long long most, long long slots) {
  int c = 1;
  while (c < 8 && (row_bytes / c > most || (rows * 2 * c <= slots && row_bytes / (2 * c) >= 8 * 1024)))
    c *= 2;
  return c;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kern)(KArgs...), long long rows, int ctas, int threads, size_t smem,
                        cudaStream_t st, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  const long long most = (1LL << 30) / ctas;
  cfg.gridDim = dim3((unsigned)((rows < most ? rows : most) * ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

}  // namespace ret
