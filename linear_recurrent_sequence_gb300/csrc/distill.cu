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
// Log probabilities that add up to more than 1 (rounded or scaled ones), or those
// of all V tokens, leave no p_r that makes up for it: with P = sum p the loss is
// T^2 (P - 1) more, and P q_j takes the place of q_j in its gradient.
//
// Bound by memory: the loss reads each logit once, the gradient reads it and
// writes a value.  bf16, a list of 64: the loss of 1024 x 65536 27.6 us, 4.9 TB/s;
// the gradient of 2048 x 65536 89.5 us, 6.0 TB/s; both of 4096 x 65536 199 us, 5.4
// TB/s (with a second reading from the L2 instead of shared memory 262 us); 8 x
// 32768 6.1 us, latency.  fp32: the loss of 1024 x 50001 44.5 us, 4.6 TB/s, both of
// 1500 x 50001 131 us, 4.6 TB/s.
//
// Eight warps of a CTA walk over its slice of the row while a ninth reads the
// list, gathers its logits and forms the teacher's probabilities; the listed
// logits' own softmax joins the others', so that the gradient can start at once
// while the ninth warp adds up the loss.  The walk waits for the list's bits:
// clearing them while the ids are on their way, and not before, made 210 us of
// loss and gradient into 195.
#include "launch.h"
#include "logits.cuh"

namespace ret {

namespace {

constexpr int kUnroll = 4;
constexpr int kMaxTop = RETNET_MAX_TOP;

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kThreads = kRowThreads + 32;  // and the list's warp
constexpr int kRowBits = 65536;             // tokens up to which the row has its bits
constexpr int kPer = kMaxTop / 32;          // its entries a lane: lane + 32 i

// The list of a row.
struct ListShared {
  alignas(16) int id[kMaxTop];  // the token, or -1: absent, out of range, listed before
  float x[kMaxTop];     // the student's logit
  float p[kMaxTop];     // the teacher's probability and its logarithm
  float ln_p[kMaxTop];
  int outside, no_teacher;
  float p_rest, over;   // over: sum p + p_rest - 1
  Softmax top;          // of the listed logits
  Softmax parts[kRowWarps], mine;
};

// p ln(p / q) - p + q from ln p and ln q.  Near p = q the difference of the
// logarithms d gives p (d - 1 + e^-d) by its series, exact to 2^-24 for |d| < 1/2;
// where q is over e^8 times p (and e^-d may be beyond fp32) q itself is added.
__device__ __forceinline__ float loss_term(float p, float ln_p, float ln_q) {
  if (p == 0.f) return expf(ln_q);
  const float d = ln_p - ln_q;
  if (d < -8.f) return fmaf(p, d - 1.f, expf(ln_q));
  float g;
  if (fabsf(d) < 0.5f) {
    g = 1.f / 2.f - d * (1.f / 6.f - d * (1.f / 24.f - d * (1.f / 120.f - d * (1.f / 720.f - d * (1.f / 5040.f - d * (1.f / 40320.f - d * (1.f / 362880.f)))))));
    g *= d * d;
  } else {
    g = d + expm1f(-d);
  }
  return __fmul_rn(p, g);  // (no contraction: the same bits wherever this is inlined)
}

// A bit for each token of the row, or of the CTA's slice alone where those of
// the row would leave fewer CTAs an SM (1500 x 131072 bf16, loss and gradient:
// 152 us, with the row's 195).  The row's own tell whether a token is listed
// twice, which the list warp has to look for otherwise (4096 x 65536 2 us more).  Vector v of the row has the kVec bits from (v - v0 +
// 1) kVec, v0 the slice's first or 0.
struct ListBits {
  unsigned *words;
  int n, v0;
  bool row;
  template <typename T>
  __device__ __forceinline__ ListBits(unsigned *w, int count, const LogitRow<T> &r, const RowSlice &slice)
      : words(w), n(count), v0(0), row(count * 32 >= r.V + 2 * LogitRow<T>::kVec) {
    if (!row) v0 = slice.v0;
  }
  // Where token i has its bit.
  template <typename T>
  __device__ __forceinline__ int at(const LogitRow<T> &r, int i) const {
    return i - r.index(v0) + LogitRow<T>::kVec;
  }
  // Masks the listed tokens of vector v.
  template <typename T>
  __device__ __forceinline__ void hide(int v, LogitVec<T> &x) const {
    constexpr int kVec = LogitRow<T>::kVec;
    const uint8_t *bytes = reinterpret_cast<const uint8_t *>(words);
    const int n = v - v0 + 1;
    const unsigned hit = kVec == 8 ? bytes[n] : (bytes[n >> 1] >> (4 * (n & 1))) & 15u;
    if (hit)
      for (int e = 0; e < kVec; ++e)
        if (hit >> e & 1u) x.mask(e);
  }
  // The logit of token i, -infinity where it is listed (or i negative).
  template <typename T>
  __device__ __forceinline__ float unlisted(const LogitRow<T> &r, int i) const {
    const int b = at(r, i);
    return i >= 0 && !(words[b >> 5] >> (b & 31) & 1u) ? logit_of(r.p[i]) : -INFINITY;
  }
};

// The list warp: the tokens of row r and their bits.  each(i, id) for the
// lane's entries; outside: one of them is past the vocabulary; repeated: one of
// them may be listed twice.
template <typename T, typename F>
__device__ __forceinline__ void read_ids(const DistillArgs &a, long long r, const LogitRow<T> &row,
                                         const RowSlice &slice, const ListBits &bits, ListShared &sh,
                                         bool &outside, bool &repeated, F each) {
  const int lane = threadIdx.x & 31;
  long long v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long k = r * a.top + lane + 32 * i;
    v[i] = -1;
    if (lane + 32 * i < a.top)
      v[i] = a.id64 ? reinterpret_cast<const long long *>(a.ids)[k] : (long long)reinterpret_cast<const int *>(a.ids)[k];
  }
  // (while the ids are on their way)
  for (int i = lane; i < bits.n / 4; i += 32) reinterpret_cast<uint4 *>(bits.words)[i] = make_uint4(0, 0, 0, 0);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    outside |= v[i] >= a.V;
    const int id = v[i] >= 0 && v[i] < a.V ? (int)v[i] : -1;
    sh.id[lane + 32 * i] = id;
    each(i, id);
    if (id >= 0 && (bits.row || slice.has(row, id))) {
      const int at = bits.at(row, id);
      repeated |= (atomicOr(&bits.words[at >> 5], 1u << (at & 31)) >> (at & 31) & 1u) != 0;
    }
  }
}

// The list warp: of a token that is listed more than once the first entry counts.
__device__ __forceinline__ void drop_repeated(const DistillArgs &a, ListShared &sh) {
  const int lane = threadIdx.x & 31;
  bool again[kPer] = {};
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (32 * i >= a.top) break;
    const int id = sh.id[lane + 32 * i];
    again[i] = (__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1)) != 0;
    for (int j = 0; j < 32 * i; j += 4) {
      const int4 q = *reinterpret_cast<const int4 *>(sh.id + j);
      again[i] |= q.x == id || q.y == id || q.z == id || q.w == id;
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (again[i]) sh.id[lane + 32 * i] = -1;
  __syncwarp();
}

// The list warp: the listed logits x (-infinity where there is none) and their
// softmax.
__device__ __forceinline__ void listed_softmax(const DistillArgs &a, ListShared &sh, const float (&x)[kPer]) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, z = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    sh.x[lane + 32 * i] = x[i];
    bad |= !(x[i] <= kFltMax);
    m = fmaxf(m, x[i]);
  }
  m = redux_max(m);
  const float mm = m > -INFINITY ? m : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) z += ex2((x[i] - mm) * a.scale);
  z = warp_sum(z);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) sh.top = {m, z, 0.f, bad};
}

// A sum in two floats: hi + lo, |lo| below an ulp of hi (Knuth's exact sum of
// two floats for each term).
struct TwoFloat {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
    hi = t;
  }
  // e^v for v > -80: with v log2(e) = n + r in two floats and z = r ln 2, the
  // three parts 2^n, 2^n z and 2^n (e^z - 1 - z), the last by its series
  // (|z| < 0.35).  Relative to e^v the error is up to 2^-26 for v > -1 and 2^-22
  // far below (z's low part is not multiplied by the series), where e^v itself is
  // small: absolutely it stays below 2^-26.6, which is what 1 - sum p needs.
  __device__ __forceinline__ void add_exp(float v) {
    constexpr float kLog2e = 1.44269502f, kLog2eLo = 1.92596303e-8f;  // log2(e) in two floats
    constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;    // ln 2
    const float t = __fmul_rn(v, kLog2e), t_lo = fmaf(v, kLog2eLo, fmaf(v, kLog2e, -t));
    const float n = rintf(t), r = __fsub_rn(t, n);
    const float z = __fmul_rn(r, kLn2);
    const float z_lo = __fadd_rn(fmaf(r, kLn2, -z), fmaf(r, kLn2Lo, __fmul_rn(t_lo, kLn2)));
    const float q = z * z * (1.f / 2.f + z * (1.f / 6.f + z * (1.f / 24.f + z * (1.f / 120.f + z * (1.f / 720.f + z * (1.f / 5040.f))))));
    const float s = exp2f(n);
    add(s);
    add(__fmul_rn(s, z));
    add(__fmul_rn(s, fmaf(z_lo, 1.f + z, q)));
  }
};

// The list warp: the teacher's probabilities.
__device__ __forceinline__ void teacher(const DistillArgs &a, float (&v)[kPer], ListShared &sh) {
  const int lane = threadIdx.x & 31;
  float p[kPer], m = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (sh.id[lane + 32 * i] < 0) v[i] = -INFINITY;
    m = max_nan(m, v[i]);
  }
  float ln_sum = 0.f;
  if (!a.tail) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    const bool none = m == -INFINITY;  // no probabilities: the row counts for nothing
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = none ? -INFINITY : __fmul_rn(v[i] - m, a.inv_t);
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
  float rest = 0.f, over = 0.f;
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
    if (rest < 0.f || listed == a.V) {  // NaN stays NaN
      over = -rest;
      rest = 0.f;
    }
  }
  if (lane == 0) {
    sh.p_rest = rest;
    sh.over = over;
  }
}

// What a row's threads need of it: ln q_j = ((x_j - a) log2(e) / T - b) ln 2, and
// with a_rest, b_rest in place of a, b  ln (q_j / q_rest), each relative to its
// own maximum; c = T w and c_rest = T w p_rest.
struct RowConstants {
  float a, b, a_rest, b_rest, c, c_rest;
  bool bad, empty;
};

// The softmax of all tokens from that of those not listed and the listed ones'.
__device__ __forceinline__ Softmax whole_row(const Softmax &rest, const Softmax &top, float scale) {
  const float m = fmaxf(rest.m, top.m), to = m > -INFINITY ? m : 0.f;
  const float z = fmaf(rest.s, ex2((rest.m - to) * scale), __fmul_rn(top.s, ex2((top.m - to) * scale)));
  return {m, z, 0.f, rest.bad || top.bad};
}

// From the softmax of all tokens and that of those not listed.
__device__ __forceinline__ RowConstants row_constants(const DistillArgs &a, float weight, const Softmax &all,
                                                      const Softmax &rest, const ListShared &sh) {
  RowConstants k;
  k.bad = all.bad || sh.outside;
  k.empty = all.m == -INFINITY;
  k.a = k.empty ? 0.f : all.m;
  k.b = k.empty ? 0.f : log2f(all.s);
  const bool none = sh.no_teacher || (k.empty && !k.bad), some = rest.s > 0.f;
  k.a_rest = some ? rest.m : 0.f;
  k.b_rest = some ? log2f(rest.s) : 0.f;
  const float w = weight * a.t;
  k.c = k.bad ? nan_value() : none ? 0.f : w;
  k.c_rest = none || !some ? 0.f : w * sh.p_rest;
  return k;
}

// The saved statistics are fp32 numbers of the size of x / T, and their rounding
// is a relative error of q: 2^-16 for those up to 256, the largest that are used.
// Beyond (a level, a finite mask, a low temperature) the row is walked over
// before its gradient, as for loss and gradient together: 2048 x 65536 bf16 170
// us where all rows are such, with the rest bucket 254 (90 and 95 us else).
constexpr float kSavedMost = 256.f;

// (NaN: a row that has no distribution, known from them.)
template <bool kTail>
__device__ __forceinline__ bool saved_too_coarse(float lse, float lse_rest, const ListShared &sh) {
  if (lse != lse) return false;
  return !(fabsf(lse) <= kSavedMost) || (kTail && sh.p_rest > 0.f && !(fabsf(lse_rest) <= kSavedMost));
}

// From the statistics that the forward saved.
__device__ __forceinline__ RowConstants saved_constants(const DistillArgs &a, float lse, float lse_rest, float weight,
                                                        bool outside, bool no_teacher, float p_rest) {
  RowConstants k;
  const float w = weight * a.t;
  const bool none = no_teacher || lse == -INFINITY;
  const bool no_rest = none || lse_rest == -INFINITY;
  // a: a level near the row's logits; b: what its rounding left out
  constexpr float kLog2e = 1.4426950408889634f;
  k.a = none ? 0.f : lse * a.t;
  k.b = none ? 0.f : -fmaf(k.a, a.inv_t, -lse) * kLog2e;
  k.a_rest = no_rest ? 0.f : lse_rest * a.t;
  k.b_rest = no_rest ? 0.f : -fmaf(k.a_rest, a.inv_t, -lse_rest) * kLog2e;
  k.c = outside ? nan_value() : none ? 0.f : w;
  k.c_rest = no_rest ? 0.f : w * p_rest;
  return k;
}

// The list warp: the row's loss and statistics.
__device__ __forceinline__ void row_loss(const DistillArgs &a, long long r, const Softmax &rest,
                                         const RowConstants &c, const ListShared &sh) {
  const int lane = threadIdx.x & 31;
  constexpr float kLn2 = 0.6931471805599453f;
  const float ln_z = __fmul_rn(c.b, kLn2);
  const float ln_qr = rest.s > 0.f ? fmaf(rest.m - c.a, a.inv_t, fmaf(c.b_rest, kLn2, -ln_z)) : -INFINITY;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int k = lane + 32 * i;
    if (k < a.top && sh.id[k] >= 0)
      sum += loss_term(sh.p[k], sh.ln_p[k], c.empty ? -INFINITY : fmaf(sh.x[k] - c.a, a.inv_t, -ln_z));
  }
  sum = warp_sum(sum);
  if (lane == 0) {
    const float pr = sh.p_rest;
    sum += loss_term(pr, logf(pr), c.empty ? -INFINITY : ln_qr);
    sum += sh.over;
    if (a.loss) a.loss[r] = c.bad ? nan_value() : sh.no_teacher ? 0.f : sum * (a.t * a.t);
    if (a.stats) {
      const bool bad = rest.bad || sh.top.bad;
      a.stats[2 * r] = bad ? nan_value() : c.empty ? -INFINITY : fmaf(c.a, a.inv_t, ln_z);
      a.stats[2 * r + 1] = bad ? nan_value() : fmaf(c.a, a.inv_t, ln_qr + ln_z);
    }
  }
}

// The gradient of a token that is not listed; total: sum p + p_rest.
struct RestGradient {
  float a, b, a_rest, b_rest, c, c_rest, scale;
  __device__ __forceinline__ RestGradient(const RowConstants &k, float sc, float total)
      : a(-k.a), b(-k.b), a_rest(-k.a_rest), b_rest(-k.b_rest), c(k.c * total), c_rest(-k.c_rest), scale(sc) {}
  template <bool kTail>
  __device__ __forceinline__ float2 at(float2 x) const {
    const float2 s2 = make_float2(scale, scale);
    const float2 q = tc::fma2(tc::add2(x, make_float2(a, a)), s2, make_float2(b, b));
    float2 g = tc::mul2(make_float2(c, c), make_float2(ex2(q.x), ex2(q.y)));
    if (kTail) {
      const float2 o = tc::fma2(tc::add2(x, make_float2(a_rest, a_rest)), s2, make_float2(b_rest, b_rest));
      g = tc::fma2(make_float2(c_rest, c_rest), make_float2(ex2(o.x), ex2(o.y)), g);
    }
    return g;
  }
};

// The CTA's slice of a row in shared memory, a thread's own vectors at
// [vector][thread]: only the thread that copied one reads it.  The copies are
// kGroups groups of kUnroll vectors a thread.
constexpr int kGroups = 4;
constexpr int kSliceBytes = kGroups * kUnroll * kRowThreads * 16;

template <typename T>
struct StagedSlice {
  uint8_t *slot;
  __device__ __forceinline__ StagedSlice(uint8_t *base) : slot(base + threadIdx.x * 16) {}
  __device__ __forceinline__ void copy(const LogitRow<T> &row, const RowSlice &slice) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int n = g * kUnroll + j, at = slice.v0 + threadIdx.x + n * kRowThreads;
        if (at < slice.v1)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(slot + n * kRowThreads * 16)),
                       "l"(row.p + row.index(at))
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // Groups 0 .. g have arrived.
  template <int g>
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1 - g) : "memory");
  }
  __device__ __forceinline__ void get(int n, LogitVec<T> &v) const {
    v.raw = *reinterpret_cast<const decltype(v.raw) *>(slot + n * kRowThreads * 16);
  }
};

// The eight warps: the gradient of the CTA's slice of the row, from the logits
// in shared memory (kStaged) or from x itself (whose first group is in
// `ahead`); x may be dx.
template <typename T, bool kTail, bool kStaged>
__device__ __forceinline__ void write_gradient(const LogitRow<T> &row, const RowSlice &slice,
                                               const StagedSlice<T> &staged, T *dx, bool zero,
                                               const RestGradient &rest, const LogitVec<T> *ahead) {
  constexpr int kVec = LogitRow<T>::kVec;
  const int tid = threadIdx.x;
  const bool vec = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(row.p)) & 15) == 0;
  auto put = [&](int at, LogitVec<T> &v) {
    float f[kVec];
    if (zero) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) f[e] = 0.f;
    } else {
      v.get(f);
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const float2 g = rest.template at<kTail>(make_float2(f[e], f[e + 1]));
        f[e] = g.x;
        f[e + 1] = g.y;
      }
    }
    T *o = dx + row.index(at);
    if (vec) {
      v.set(f);
      v.store(o);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        Elems<T, 1> one;
        const float g1[1] = {f[e]};
        one.set(g1);
        one.store(o + e);
      }
    }
  };
  int i = slice.v0 + tid;
  if (kStaged) {
    for (int n = 0; i < slice.v1; i += kRowThreads, ++n) {
      LogitVec<T> v;
      staged.get(n, v);
      put(i, v);
    }
  } else {
    if (ahead) {
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (i + j * kRowThreads < slice.v1) {
          LogitVec<T> v = ahead[j];
          put(i + j * kRowThreads, v);
        }
      i += kUnroll * kRowThreads;
    }
    for (; i + (kUnroll - 1) * kRowThreads < slice.v1; i += kUnroll * kRowThreads) {
      LogitVec<T> v[kUnroll];
      if (!zero)
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) v[j].load(row.p + row.index(i + j * kRowThreads));
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) put(i + j * kRowThreads, v[j]);
    }
    for (; i < slice.v1; i += kRowThreads) {
      LogitVec<T> v;
      if (!zero) v.load(row.p + row.index(i));
      put(i, v);
    }
  }
  const int single = slice.single(row);
  if (single >= 0) {
    const float x = zero ? 0.f : logit_of(row.p[single]);
    const float g1[1] = {zero ? 0.f : rest.template at<kTail>(make_float2(x, x)).x};
    Elems<T, 1> one;
    one.set(g1);
    one.store(dx + single);
  }
}

// The softmax of the row's tokens (kRest: of those that are not listed), by all
// of its CTAs' threads, a vector at a time: for the few rows whose saved
// statistics do not serve.
template <typename T, bool kRest>
__device__ __forceinline__ Softmax walk_again(const LogitRow<T> &row, const RowSlice &slice, const ListBits &bits,
                                              float scale, uint32_t ctas, ListShared &sh) {
  Softmax part = {-INFINITY, 0.f, 0.f, 0};
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < kRowThreads) {
    const Scale sc(scale);
    WarpSoftmax acc;
#pragma unroll 1
    for (int i = slice.v0 + (tid & ~31); i < slice.v1; i += kRowThreads) {
      LogitVec<T> v[1];
      v[0].fill_masked();
      if (i + lane < slice.v1) {
        v[0].load(row.p + row.index(i + lane));
        if (kRest) bits.hide(i + lane, v[0]);
      }
      acc.group<T, 1, false>(v, sc);
    }
    if (tid < 32) {
      const int single = slice.single(row);
      acc.single<false>(kRest ? bits.unlisted(row, single) : single >= 0 ? logit_of(row.p[single]) : -INFINITY, sc);
    }
    part = acc.all<false>(sc);
  }
  const Softmax all = join_row<false, kRowWarps>(part, scale, ctas, sh.parts, &sh.mine);
  if (ctas > 1) {
    cluster_have_read();
    cluster_wait_read();
  }
  __syncthreads();
  return all;
}

// The eight warps: the slice of the row filled with one value.
template <typename T>
__device__ __forceinline__ void fill_slice(const LogitRow<T> &row, const RowSlice &slice, T *dx, float x) {
  const int i0 = slice.first ? 0 : row.index(slice.v0), i1 = slice.last ? row.V : row.index(slice.v1);
  Elems<T, 1> one;
  const float g1[1] = {x};
  one.set(g1);
  for (int i = i0 + threadIdx.x; i < i1; i += kRowThreads) one.store(dx + i);
}

// Barrier 1: the list is ready.  (Its warp waits too, which orders its shared
// memory for the others; to arrive after a fence instead would wait for all of
// its loads.)
__device__ __forceinline__ void list_ready() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// CTAs an SM: three where their slices fill its shared memory, four for the
// gradient alone, six for the loss alone (1024 x 65536 bf16 27.4 us, with four
// 33.8; the 32 registers that six leave spill 40 to 52 bytes a thread, the 56 of
// four up to 32).
template <typename T, int kWhat, bool kTail, bool kStaged>
__global__ void __launch_bounds__(kThreads, kStaged ? 3 : kWhat == kDistillFwd ? 6 : 4)
distill_kernel(const DistillArgs a, int words) {
  constexpr bool kFwd = (kWhat & kDistillFwd) != 0, kBwd = (kWhat & kDistillBwd) != 0;
  extern __shared__ __align__(16) uint8_t dyn[];  // the bits, then the staged slice
  __shared__ ListShared sh;
  pdl_launch_dependents();
  pdl_wait();
  StagedSlice<T> staged(dyn + (size_t)words * 4);
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  const bool walks = tid < kRowThreads;
  for (long long r = blockIdx.x / ctas; r < a.rows; r += gridDim.x / ctas) {
    const LogitRow<T> row(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), a.V);
    const RowSlice slice(row, ctas, rank);
    const ListBits bits(reinterpret_cast<unsigned *>(dyn), words, row, slice);
    T *dx = kBwd ? reinterpret_cast<T *>(a.dx) + row_offset(a.sd, r) : nullptr;
    const float weight = kBwd && a.weight ? a.weight[r] : 1.f;
    const bool zero = kBwd && weight == 0.f;
    if (!kFwd && zero) {
      if (walks) write_gradient<T, kTail, false>(row, slice, staged, dx, true, RestGradient({}, 0.f, 1.f), nullptr);
      continue;
    }
    // (asked for before the logits, so that they are there with the list)
    const float lse = kFwd ? 0.f : a.stats[2 * r], lse_rest = kFwd || !kTail ? -INFINITY : a.stats[2 * r + 1];
    Softmax part = {-INFINITY, 0.f, 0.f, 0};
    LogitVec<T> ahead[kStaged ? 1 : kUnroll];  // the first group, on its way while the list is read
    int i = slice.v0 + (tid & ~31);            // of the warp's first lane: the loops are the warp's
    if (!walks) {
      float values[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        values[j] = lane + 32 * j < a.top ? a.values[r * a.top + lane + 32 * j] : -INFINITY;
      // The listed logits: for the loss after the list is ready, which the walk
      // waits for (before: 4096 x 65536 bf16, loss and gradient, 205 us, so 197);
      // for the gradient alone at once (2048 x 65536: 89 us, later 92), and only
      // those of the CTA's own slice: where it is written over the logits,
      // another CTA may be past its slice already.
      T raw[kPer];
      auto gather = [&](int j, int id) {
        raw[j] = T(-INFINITY);
        if (id >= 0 && (kFwd || slice.has(row, id))) raw[j] = row.p[id];
      };
      bool outside = false, repeated = !bits.row;
      read_ids(a, r, row, slice, bits, sh, outside, repeated, [&](int j, int id) {
        if (!kFwd) gather(j, id);
      });
      if (kFwd) list_ready();
      outside = __any_sync(0xffffffffu, outside);
      if (lane == 0) sh.outside = outside;
      if (__any_sync(0xffffffffu, repeated)) drop_repeated(a, sh);
      float x[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int id = sh.id[lane + 32 * j];
        if (kFwd) gather(j, id);
        x[j] = id >= 0 ? logit_of(raw[j]) : -INFINITY;
      }
      listed_softmax(a, sh, x);
      // (the gradient alone may be written over the logits: only from here on)
      if (!kFwd && !kTail) list_ready();
      teacher(a, values, sh);
      if (!kFwd && kTail) list_ready();
    } else {
      if (kStaged) {
        staged.copy(row, slice);
      } else {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
          const int at = i + lane + j * kRowThreads;
          if (at < slice.v1)
            ahead[kStaged ? 0 : j].load(row.p + row.index(at));
          else
            ahead[kStaged ? 0 : j].fill_masked();
        }
      }
      list_ready();  // for the bits; for the gradient alone: its logits, with the rest bucket p_rest
      if (kFwd) {
        // the softmax of the tokens that are not listed
        const Scale sc(a.scale);
        WarpSoftmax acc;
        // One group of vectors, from slots n.. (kStaged), from `ahead` or from the row.
        auto group = [&](int n, bool first) {
          if (i >= slice.v1) return;
          LogitVec<T> v[kUnroll];
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) {
            const int at = i + lane + j * kRowThreads;
            const bool in = at < slice.v1;
            if (!kStaged && first)
              v[j] = ahead[kStaged ? 0 : j];
            else if (!in)
              v[j].fill_masked();
            else if (kStaged)
              staged.get(n + j, v[j]);
            else
              v[j].load(row.p + row.index(at));
          }
#pragma unroll
          for (int j = 0; j < kUnroll; ++j)
            if (i + lane + j * kRowThreads < slice.v1) bits.hide(i + lane + j * kRowThreads, v[j]);
          acc.group<T, kUnroll, false>(v, sc);
          i += kUnroll * kRowThreads;
        };
        if (kStaged) {
          staged.template wait<0>();
          group(0, false);
          staged.template wait<1>();
          group(kUnroll, false);
          staged.template wait<2>();
          group(2 * kUnroll, false);
          staged.template wait<3>();
          group(3 * kUnroll, false);
        } else {
          group(0, true);
          while (i < slice.v1) group(0, false);
        }
        if (tid < 32) acc.single<false>(bits.unlisted(row, slice.single(row)), sc);
        part = acc.all<false>(sc);
      }
    }
    RowConstants k;
    if (kFwd) {
      const Softmax rest = join_row<false, kRowWarps>(part, a.scale, ctas, sh.parts, &sh.mine);
      if (ctas > 1) cluster_have_read();
      if (kBwd || !walks) k = row_constants(a, weight, whole_row(rest, sh.top, a.scale), rest, sh);
      if (!walks && rank == 0) row_loss(a, r, rest, k, sh);
    } else if (saved_too_coarse<kTail>(lse, lse_rest, sh)) {
      // (the same in all CTAs of the row; nothing has been written over it yet)
      const Softmax all = walk_again<T, false>(row, slice, bits, a.scale, ctas, sh);
      Softmax rest = {-INFINITY, 0.f, 0.f, 0};
      if (kTail) rest = walk_again<T, true>(row, slice, bits, a.scale, ctas, sh);
      k = row_constants(a, weight, all, rest, sh);
    } else {
      if (walks && !kTail)
        k = saved_constants(a, lse, lse_rest, weight, sh.outside, false, 0.f);  // the teacher is looked at below
      else
        k = saved_constants(a, lse, lse_rest, weight, sh.outside, sh.no_teacher, sh.p_rest);
    }
    if (kBwd) {
      if (walks)
        write_gradient<T, kTail, kStaged>(row, slice, staged, dx, zero,
                                          RestGradient(k, a.scale, kTail ? 1.f + sh.over : 1.f),
                                          kFwd || kStaged ? nullptr : ahead);
      __syncthreads();
      // A row without a teacher, where the gradient did not wait to know it.
      const bool blank = !kFwd && !kTail && sh.no_teacher && !sh.outside && lse == lse;
      if (blank && walks) fill_slice(row, slice, dx, 0.f);
      // The listed tokens' gradients replace what stands there; each is written
      // by the CTA whose slice it is in.
      if (!walks && !zero) {
        const float total = kTail ? 1.f + sh.over : 1.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int id = sh.id[lane + 32 * j];
          if (id >= 0 && slice.has(row, id) && !blank) {
            const float q = ex2(fmaf(sh.x[lane + 32 * j] - k.a, a.scale, -k.b));
            const float g1[1] = {k.c * fmaf(total, q, -sh.p[lane + 32 * j])};
            Elems<T, 1> one;
            one.set(g1);
            one.store(dx + id);
          }
        }
      }
    }
    // the row's list has been read, its part of the softmax by the other CTAs too
    if (ctas > 1 && kFwd) cluster_wait_read();
    __syncthreads();
  }
}

template <typename T, int kWhat, bool kTail, bool kStaged>
cudaError_t launch_as(const DistillArgs &a, int ctas, size_t smem, int words, cudaStream_t st) {
  auto kern = distill_kernel<T, kWhat, kTail, kStaged>;
  static std::atomic<unsigned> done{0};
  if (smem > 32 * 1024) {
    const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
    if (e != cudaSuccess) return e;
  }
  return launch_rows(kern, a.rows, ctas, kThreads, smem, st, a, words);
}

template <typename T, int kWhat>
cudaError_t launch(const DistillArgs &a, cudaStream_t st) {
  constexpr int kVec = LogitRow<T>::kVec;
  const long long row_bytes = (long long)a.V * sizeof(T);
  const int sms = device_sms();
  // A slice that fits in shared memory while a cluster of 8 can share the row
  // (loss and gradient together; the loss alone has the same slices, so that
  // both calls give the same bits).
  int ctas = row_ctas(a.rows, row_bytes, kWhat == kDistillBwd ? 1LL << 40 : kSliceBytes,
                      (kWhat == kDistillBwd ? 4LL : 3LL) * sms);
  const int vecs = (a.V / kVec + ctas - 1) / ctas;  // of a slice
  auto words_of = [](int tokens) { return ((tokens + 2 * kVec + 31) / 32 + 3) / 4 * 4; };
  const int words = words_of(a.V <= kRowBits ? a.V : vecs * kVec);
  const size_t bits = (size_t)words * 4;
  if constexpr (kWhat == kDistillStep) {
    if (vecs * 16 <= kSliceBytes) {
      const size_t smem = bits + (size_t)((vecs + kRowThreads - 1) / kRowThreads) * kRowThreads * 16;
      return a.tail ? launch_as<T, kDistillStep, true, true>(a, ctas, smem, words, st)
                    : launch_as<T, kDistillStep, false, true>(a, ctas, smem, words, st);
    }
  }
  return a.tail ? launch_as<T, kWhat, true, false>(a, ctas, bits, words, st)
                : launch_as<T, kWhat, false, false>(a, ctas, bits, words, st);
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
