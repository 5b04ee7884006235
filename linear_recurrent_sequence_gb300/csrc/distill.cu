// Distillation of a student's logits x [rows][V] from a teacher's list of at
// most 128 tokens a row, at temperature T.  With q = softmax(x / T), p_k the
// teacher's probability of the row's k-th token and p_r what it leaves to
// all other tokens (q_r likewise):
//   L = T^2 [ sum_k f(p_k, q_k) + f(p_r, q_r) ],  f(p, q) = p ln(p / q) - p + q,
//   dL/dx_j = T (q_j - p_j) for the listed, T (q_j - p_r q_j / q_r) for the others.
// Without the rest bucket p is the softmax of the list alone and p_r = 0.
// Since sum p + p_r = sum q + q_r = 1, L is T^2 times the divergence
// sum p ln(p / q); its terms are never negative, so that a small loss is not
// the difference of large ones.  q_r is summed over the tokens that are not
// listed (a bit per token in shared memory tells which), not taken as
// 1 - sum q_k.
//
// Bound by memory: the loss reads each logit once, the gradient reads it and
// writes a value.  Loss and gradient in one call: the second reading of the
// row finds it in L2.
#include "launch.h"
#include "logits.cuh"

namespace ret {

namespace {

constexpr int kThreads = 512;
constexpr int kUnroll = 4;
constexpr int kMaxTop = RETNET_MAX_TOP;

// The list of a row and the row's constants.
struct ListShared {
  int id[kMaxTop];      // the token, or -1: absent, out of range, listed before
  float x[kMaxTop];     // the student's logit
  float p[kMaxTop];     // the teacher's probability and its logarithm
  float ln_p[kMaxTop];
  int repeated, outside, no_teacher;
  float p_rest;
  // ln q_j = ((x_j - a) log2(e) / T - b) ln 2, and with a_rest, b_rest in
  // place of a, b  ln (q_j / q_rest): each relative to its own maximum
  float a, b, a_rest, b_rest;
  float c, c_rest;      // T w and T w p_rest
  Softmax joined[kThreads / 32];
};

__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fffffff); }

// p ln(p / q) - p + q from ln p and ln q.  Near p = q the difference of the
// logarithms d gives p (d - 1 + e^-d) by its series, exact to 2^-24 for |d| < 1/2.
__device__ __forceinline__ float loss_term(float p, float ln_p, float ln_q) {
  if (p == 0.f) return expf(ln_q);
  const float d = ln_p - ln_q;
  float g;
  if (fabsf(d) < 0.5f) {
    g = 1.f / 2.f - d * (1.f / 6.f - d * (1.f / 24.f - d * (1.f / 120.f - d * (1.f / 720.f - d * (1.f / 5040.f - d * (1.f / 40320.f - d * (1.f / 362880.f)))))));
    g *= d * d;
  } else {
    g = d + expm1f(-d);
  }
  return p * g;
}

// The tokens of row r: validity, the bit of each in `bits`, the student's
// logits.  Bit position of token i: i - head + kVec, so that vector v of the
// row has the kVec bits from (v + 1) kVec.
template <typename T>
__device__ __forceinline__ void read_list(const DistillArgs &a, long long r, const LogitRow<T> &row,
                                          unsigned *bits, int words, ListShared &sh) {
  constexpr int kVec = LogitRow<T>::kVec;
  for (int i = threadIdx.x; i < words; i += kThreads) bits[i] = 0u;
  if (threadIdx.x == 0) sh.repeated = sh.outside = 0;
  __syncthreads();
  const int k = threadIdx.x;
  int id = -1;
  if (k < a.top) {
    const long long v = a.id64 ? reinterpret_cast<const long long *>(a.ids)[r * a.top + k]
                               : (long long)reinterpret_cast<const int *>(a.ids)[r * a.top + k];
    if (v >= a.V) sh.outside = 1;
    if (v >= 0 && v < a.V) {
      id = (int)v;
      const int at = id - row.head + kVec;
      if (atomicOr(&bits[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u) sh.repeated = 1;
    }
    sh.id[k] = id;
  }
  __syncthreads();
  if (sh.repeated && k < a.top && id >= 0)
    for (int j = 0; j < k; ++j)
      if (sh.id[j] == id) id = -1;
  if (sh.repeated) {
    __syncthreads();
    if (k < a.top) sh.id[k] = id;
  }
  if (k < a.top) sh.x[k] = id >= 0 ? logit_of(row.p[id]) : -INFINITY;
  __syncthreads();
}

// A sum in two floats: hi + lo, |lo| below an ulp of hi.
struct TwoFloat {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float t = hi + x, b = t - hi;
    lo += (hi - (t - b)) + (x - b);
    hi = t;
  }
  // e^v for v > -80, to about 2^-28 of it: with v log2(e) = n + r in two
  // floats and z = r ln 2, the three parts 2^n, 2^n z and 2^n (e^z - 1 - z),
  // the last by its series (|z| < 0.35).
  __device__ __forceinline__ void add_exp(float v) {
    constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-8f;  // log2(e) in two floats
    constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;    // ln 2
    const float t = v * kLog2e, t_lo = fmaf(v, kLog2eLo, fmaf(v, kLog2e, -t));
    const float n = rintf(t), r = t - n;
    const float z = r * kLn2, z_lo = fmaf(r, kLn2, -z) + fmaf(r, kLn2Lo, t_lo * kLn2);
    const float q = z * z * (1.f / 2.f + z * (1.f / 6.f + z * (1.f / 24.f + z * (1.f / 120.f + z * (1.f / 720.f + z * (1.f / 5040.f))))));
    const float s = exp2f(n);
    add(s);
    add(s * z);
    add(s * fmaf(z_lo, 1.f + z, q));
  }
};

// The teacher's probabilities (warp 0; a lane has the entries lane + 32 i).
__device__ __forceinline__ void teacher(const DistillArgs &a, long long r, ListShared &sh) {
  const int lane = threadIdx.x;
  constexpr int kPer = kMaxTop / 32;
  float v[kPer], p[kPer], m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    v[i] = k < a.top && sh.id[k] >= 0 ? a.values[r * a.top + k] : -INFINITY;
    m = max_nan(m, v[i]);
  }
  float ln_sum = 0.f;
  if (!a.tail) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    const bool none = m == -INFINITY;  // no probabilities: the row counts for nothing
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = none ? -INFINITY : (v[i] - m) * a.inv_t;
    if (lane == 0) sh.no_teacher = none;
  } else if (lane == 0) {
    sh.no_teacher = 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    p[i] = expf(v[i]);
    sum += p[i];
  }
  sum = warp_sum(sum);
  const float inv = a.tail || sum == 0.f ? 1.f : 1.f / sum;
  if (!a.tail && sum > 0.f) ln_sum = logf(sum);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < a.top) {
      sh.p[lane + 32 * i] = p[i] * inv;
      sh.ln_p[lane + 32 * i] = v[i] - ln_sum;
    }
  float rest = 0.f;
  if (a.tail) {
    // 1 - sum p is small for a teacher that is sure of its list, so the sum
    // is formed in two floats.  A list of all tokens leaves nothing.
    TwoFloat two = {0.f, 0.f};
    int listed = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int k = lane + 32 * i;
      listed += __popc(__ballot_sync(0xffffffffu, k < a.top && sh.id[k] >= 0));
      if (!(v[i] <= -80.f)) two.add_exp(v[i]);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const float hi = __shfl_xor_sync(0xffffffffu, two.hi, s);
      const float lo = __shfl_xor_sync(0xffffffffu, two.lo, s);
      two.add(hi);
      two.lo += lo;
    }
    rest = (1.f - two.hi) - two.lo;
    if (rest < 0.f || listed == a.V) rest = 0.f;  // NaN stays NaN
  }
  if (lane == 0) sh.p_rest = rest;
}

// Warp 0: the student's normaliser from the softmax `rest` of the tokens
// that are not listed and the listed logits; the row's loss and statistics.
__device__ __forceinline__ void row_loss(const DistillArgs &a, long long r, const Softmax &rest,
                                         ListShared &sh) {
  const int lane = threadIdx.x;
  constexpr int kPer = kMaxTop / 32;
  float x[kPer], m = rest.m;
  bool bad = rest.bad;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    x[i] = k < a.top && sh.id[k] >= 0 ? sh.x[k] : -INFINITY;
    bad |= !(x[i] <= 3.402823466e38f);
    m = fmaxf(m, x[i]);
  }
  m = warp_max(m);
  bad = __any_sync(0xffffffffu, bad) || sh.outside;
  const bool empty = m == -INFINITY;
  if (empty) m = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) z += ex2((x[i] - m) * a.scale);
  z = warp_sum(z);
  const float dr = rest.m - m;  // -infinity where nothing is left
  z += rest.s * ex2(dr * a.scale);
  const float ln_z = logf(z);
  const float ln_qr = rest.s > 0.f ? dr * a.inv_t + (logf(rest.s) - ln_z) : -INFINITY;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    if (k < a.top && sh.id[k] >= 0)
      sum += loss_term(sh.p[k], sh.ln_p[k], empty ? -INFINITY : (x[i] - m) * a.inv_t - ln_z);
  }
  sum = warp_sum(sum);
  const float pr = sh.p_rest;
  sum += loss_term(pr, logf(pr), empty ? -INFINITY : ln_qr);
  if (lane == 0) {
    if (a.loss) a.loss[r] = bad ? nan_value() : sh.no_teacher ? 0.f : sum * (a.t * a.t);
    if (a.stats) {
      a.stats[2 * r] = bad && !sh.outside ? nan_value() : empty ? -INFINITY : fmaf(m, a.inv_t, ln_z);
      a.stats[2 * r + 1] = bad && !sh.outside ? nan_value() : fmaf(m, a.inv_t, ln_qr + ln_z);
    }
    const float w = (a.weight ? a.weight[r] : 1.f) * a.t;
    sh.a = m;
    sh.b = empty ? 0.f : log2f(z);
    sh.a_rest = rest.s > 0.f ? rest.m : 0.f;
    sh.b_rest = rest.s > 0.f ? log2f(rest.s) : 0.f;
    const bool none = sh.no_teacher || (empty && !bad);
    sh.c = bad ? nan_value() : none ? 0.f : w;
    sh.c_rest = none || !(rest.s > 0.f) ? 0.f : w * pr;
  }
}

// The row's constants from the statistics that the forward saved.
__device__ __forceinline__ void row_constants(const DistillArgs &a, long long r, ListShared &sh) {
  const float lse = a.stats[2 * r], lse_rest = a.stats[2 * r + 1];
  const float w = (a.weight ? a.weight[r] : 1.f) * a.t;
  const bool none = sh.no_teacher || lse == -INFINITY;
  const bool no_rest = none || lse_rest == -INFINITY;
  // a: a level near the row's logits; b: what its rounding left out
  constexpr float kLog2e = 1.4426950408889634f;
  sh.a = none ? 0.f : lse * a.t;
  sh.b = none ? 0.f : -fmaf(sh.a, a.inv_t, -lse) * kLog2e;
  sh.a_rest = no_rest ? 0.f : lse_rest * a.t;
  sh.b_rest = no_rest ? 0.f : -fmaf(sh.a_rest, a.inv_t, -lse_rest) * kLog2e;
  sh.c = sh.outside ? nan_value() : none ? 0.f : w;
  sh.c_rest = no_rest ? 0.f : w * sh.p_rest;
}

// The gradient of a token that is not listed.
struct RestGradient {
  float a, b, a_rest, b_rest, c, c_rest, scale;
  __device__ __forceinline__ RestGradient(const ListShared &sh, float sc)
      : a(-sh.a), b(-sh.b), a_rest(-sh.a_rest), b_rest(-sh.b_rest), c(sh.c), c_rest(-sh.c_rest),
        scale(sc) {}
  template <bool kTail>
  __device__ __forceinline__ float2 at(float2 x) const {
    const float2 s2 = make_float2(scale, scale);
    const float2 q = tc::fma2(tc::add2(x, make_float2(a, a)), s2, make_float2(b, b));
    float2 g = make_float2(c * ex2(q.x), c * ex2(q.y));
    if (kTail) {
      const float2 o = tc::fma2(tc::add2(x, make_float2(a_rest, a_rest)), s2, make_float2(b_rest, b_rest));
      g = make_float2(fmaf(c_rest, ex2(o.x), g.x), fmaf(c_rest, ex2(o.y), g.y));
    }
    return g;
  }
};

// The gradient row; x may be dx.
template <typename T, bool kTail>
__device__ __forceinline__ void write_gradient(const DistillArgs &a, const LogitRow<T> &row, T *dx,
                                               bool zero, const ListShared &sh) {
  constexpr int kVec = LogitRow<T>::kVec;
  const int tid = threadIdx.x;
  const RestGradient rest(sh, a.scale);
  const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(row.p)) & 15) == 0;
  for (int i = tid; i < row.nvec; i += kUnroll * kThreads) {
    LogitVec<T> v[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int at = i + j * kThreads;
      if (at < row.nvec && !zero) v[j].load(row.p + row.index(at));
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int at = i + j * kThreads;
      if (at >= row.nvec) continue;
      float f[kVec];
      if (zero) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = 0.f;
      } else {
        v[j].get(f);
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const float2 g = rest.template at<kTail>(make_float2(f[e], f[e + 1]));
          f[e] = g.x;
          f[e + 1] = g.y;
        }
      }
      T *o = dx + row.index(at);
      if (vec) {
        v[j].set(f);
        v[j].store(o);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          Elems<T, 1> one;
          const float g1[1] = {f[e]};
          one.set(g1);
          one.store(o + e);
        }
      }
    }
  }
  for (int which = 0; which < 2; ++which) {
    const int i = which ? row.tail_index() + tid : tid;
    if (tid < (which ? row.tail : row.head)) {
      const float x = zero ? 0.f : logit_of(row.p[i]);
      const float g1[1] = {zero ? 0.f : rest.template at<kTail>(make_float2(x, x)).x};
      Elems<T, 1> one;
      one.set(g1);
      one.store(dx + i);
    }
  }
  if (zero) return;
  __syncthreads();  // the listed tokens' gradients replace what stands there
  if (tid < a.top && sh.id[tid] >= 0) {
    const float q = ex2(fmaf(sh.x[tid] - sh.a, a.scale, -sh.b));
    const float g1[1] = {sh.c * (q - sh.p[tid])};
    Elems<T, 1> one;
    one.set(g1);
    one.store(dx + sh.id[tid]);
  }
}

template <typename T, int kWhat, bool kTail>
__global__ void __launch_bounds__(kThreads)
distill_kernel(const DistillArgs a, int words) {
  constexpr int kVec = LogitRow<T>::kVec;
  extern __shared__ unsigned bits[];
  __shared__ ListShared sh;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const LogitRow<T> row(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), a.V);
    T *dx = (kWhat & kDistillBwd) ? reinterpret_cast<T *>(a.dx) + row_offset(a.sd, r) : nullptr;
    const bool zero = (kWhat & kDistillBwd) && a.weight && a.weight[r] == 0.f;
    if (kWhat == kDistillBwd && zero) {
      write_gradient<T, kTail>(a, row, dx, true, sh);
      continue;
    }
    read_list(a, r, row, bits, words, sh);
    if (tid < 32) teacher(a, r, sh);
    if (kWhat & kDistillFwd) {
      // the softmax of the tokens that are not listed
      const uint8_t *bytes = reinterpret_cast<const uint8_t *>(bits);
      Softmax acc = Softmax::none();
      for (int i = tid; i < row.nvec; i += kUnroll * kThreads) {
        LogitVec<T> v[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int at = i + j * kThreads;
          if (at < row.nvec)
            v[j].load(row.p + row.index(at));
          else
            v[j].fill_masked();
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int at = i + j * kThreads + 1;
          if (at <= row.nvec) {
            const unsigned hit = kVec == 8 ? bytes[at] : (bytes[at >> 1] >> (4 * (at & 1))) & 15u;
            if (hit)
              for (int e = 0; e < kVec; ++e)
                if (hit >> e & 1u) v[j].mask(e);
          }
        }
        acc.group<T, kUnroll, false>(v, a.scale);
      }
      for (int which = 0; which < 2; ++which) {
        const int i = which ? row.tail_index() + tid : tid, at = i - row.head + kVec;
        if (tid < (which ? row.tail : row.head) && !(bits[at >> 5] >> (at & 31) & 1u)) {
          const float x = logit_of(row.p[i]);
          acc.raise(x, a.scale);
          acc.take(x, a.scale);
        }
      }
      const Softmax rest = join_cta(acc, a.scale, sh.joined);
      if (tid < 32) row_loss(a, r, rest, sh);
    } else if (tid < 32) {
      __syncwarp();
      if (tid == 0) row_constants(a, r, sh);
    }
    if (kWhat & kDistillBwd) {
      __syncthreads();
      write_gradient<T, kTail>(a, row, dx, zero, sh);
    }
    __syncthreads();  // the row's list has been read
  }
}

template <typename T, int kWhat>
cudaError_t launch(const DistillArgs &a, cudaStream_t st) {
  const int words = (a.V + 2 * LogitRow<T>::kVec + 31) / 32;
  const size_t smem = (size_t)words * 4;
  auto kern = a.tail ? distill_kernel<T, kWhat, true> : distill_kernel<T, kWhat, false>;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)(a.rows < (1LL << 30) ? a.rows : (1LL << 30)));
  return launch_k(kern, grid, dim3(kThreads), smem, st, true, a, words);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, int bf16, int what, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  if (what == kDistillFwd)
    return bf16 ? launch<__nv_bfloat16, kDistillFwd>(a, st) : launch<float, kDistillFwd>(a, st);
  if (what == kDistillBwd)
    return bf16 ? launch<__nv_bfloat16, kDistillBwd>(a, st) : launch<float, kDistillBwd>(a, st);
  return bf16 ? launch<__nv_bfloat16, kDistillStep>(a, st) : launch<float, kDistillStep>(a, st);
}

}  // namespace ret
