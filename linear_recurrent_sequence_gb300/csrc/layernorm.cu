// LayerNorm over rows of d values and its gradients.
//   y = (x - mean) rstd w + b,  rstd = 1 / sqrt(var + eps), biased variance;
//   with h = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - h mean(g h)),  dw = sum_rows dy h,  db = sum_rows dy.
// fp32 arithmetic for bf16 and fp32 rows; mean, rstd, w, b, dw, db in fp32.
// Little arithmetic for the bytes: 2 (forward) or 3 (backward) row elements
// move per value and at most 13 flop are done with them.
//
// The variance is the mean square of the deviations, taken after the mean:
// a row with a large level loses nothing to cancellation.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "rows.cuh"

namespace ret {

namespace {

// Sums of N values over the `tpr` threads that share a row: a power of two up
// to 32 lanes of a warp, or whole warps that exchange through red (consecutive
// calls alternate between two buffers, so a warp that is ahead cannot
// overwrite what another still reads).  They meet at the CTA's barrier, or
// with kNamed (several row groups in a CTA) at named barrier 1 + group.  A
// kernel with named barriers reserves all 16 of a CTA, and only four such
// CTAs fit an SM.
constexpr int kRed = 128;  // 8 places a row group, or one group's 32 warps

template <int N, bool kNamed>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*red)[kRed], int tpr) {
  if (tpr < 32) {
    for (int s = tpr >> 1; s > 0; s >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], s);
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = warp_sum(x[i]);
  if (tpr == 32) return;
  const int nw = tpr >> 5, lane = threadIdx.x & 31;
  const int group = kNamed ? threadIdx.x / tpr : 0, w = (threadIdx.x - group * tpr) >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i][group * 8 + w] = x[i];
  if (kNamed)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  else
    __syncthreads();
  if (nw <= 8) {  // (places without a warp hold 0)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 p = *reinterpret_cast<const float4 *>(&red[i][group * 8]);
      const float4 q = *reinterpret_cast<const float4 *>(&red[i][group * 8 + 4]);
      x[i] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = warp_sum(lane < nw ? red[i][lane] : 0.f);
  }
}

// Zeros in the exchange buffers, before their first use.
__device__ __forceinline__ void clear_red(float *red, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
}

// VEC fp32 parameters (16-byte aligned where VEC > 1), `other` where p is
// null (kThere: it is known not to be).
template <int VEC, bool kThere = false>
__device__ __forceinline__ void load_param(const float *p, size_t c, float other, float (&f)[VEC]) {
  if (!kThere && !p) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = other;
  } else if (VEC == 1) {
    f[0] = p[c];
  } else {
#pragma unroll
    for (int j = 0; j + 3 < VEC; j += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p + c + j);
      f[j] = v.x; f[j + 1] = v.y; f[j + 2] = v.z; f[j + 3] = v.w;
    }
  }
}

// VEC values at a time as packed pairs (or one value).
template <int VEC>
struct Pairs {
  static constexpr int N = VEC > 1 ? VEC / 2 : 1;
  float2 v[N];
  __device__ __forceinline__ Pairs() {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ explicit Pairs(const float (&f)[VEC]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(f[VEC > 1 ? 2 * i : 0], VEC > 1 ? f[VEC > 1 ? 2 * i + 1 : 0] : 0.f);
  }
  __device__ __forceinline__ void put(float (&f)[VEC]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[VEC > 1 ? 2 * i : 0] = v[i].x;
      if (VEC > 1) f[VEC > 1 ? 2 * i + 1 : 0] = v[i].y;
    }
  }
};

template <int VEC>
__device__ __forceinline__ float2 padd(float2 a, float2 b) {
  return VEC > 1 ? tc::add2(a, b) : make_float2(__fadd_rn(a.x, b.x), 0.f);
}
template <int VEC>
__device__ __forceinline__ float2 pmul(float2 a, float2 b) {
  return VEC > 1 ? tc::mul2(a, b) : make_float2(__fmul_rn(a.x, b.x), 0.f);
}
template <int VEC>
__device__ __forceinline__ float2 pfma(float2 a, float2 b, float2 c) {
  return VEC > 1 ? tc::fma2(a, b, c) : make_float2(fmaf(a.x, b.x, c.x), 0.f);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The row group that a thread belongs to: its tpr threads, this thread's place
// among them, and its NV vectors of VEC values.  With whole warps a row
// (kWarps) each warp has NV * 32 neighbouring vectors, so that the steps
// between a thread's vectors are constants and at most one warp is not full
// (8001 x 4097 bf16 forward, two rows of 16: 52 us, with the group's vectors
// interleaved 74).
template <int VEC, int NV, bool kWarps>
struct RowGroup {
  int tpr, group, t, t0, left;  // left: columns from the first one on
  bool full;                    // this warp has all of its vectors
  __device__ __forceinline__ RowGroup(int threads, int d)
      : tpr(threads), group(threadIdx.x / threads), t(threadIdx.x % threads) {
    t0 = (kWarps ? t / 32 * 32 * NV + t % 32 : t) * VEC;
    left = d - t0;
    full = kWarps && __all_sync(0xffffffffu, (NV - 1) * step() < left);
  }
  __device__ __forceinline__ int step() const { return (kWarps ? 32 : tpr) * VEC; }
  __device__ __forceinline__ bool has(int i) const { return i * step() < left; }
  // f(i, whether vector i is there) for each vector; `there`: any of them is.
  template <typename F>
  __device__ __forceinline__ void each(bool there, F f) const {
    if (kWarps && full && there) {  // as in all warps but the last
#pragma unroll
      for (int i = 0; i < NV; ++i) f(i, std::true_type());
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) f(i, there && has(i));
    }
  }
};

// The rows ahead, kRows at a time, on their way through shared memory by
// asynchronous copies.  copy_row() is called by all threads of the row group
// for row n of a stage; after wait() view() gives a thread its vectors (`in`:
// the row is live and has vector i).
template <typename T, int VEC, int NV, bool kWarps, int kRows, int kStages, bool kNamed>
struct RowRing {
  // A thread copies the vectors that it reads: slots [stage][row][warp][vector]
  // [lane], and no barrier.  What is past the row's end, or of a row that is
  // not there, arrives as zeros.
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static size_t bytes(int, int threads, int) { return (size_t)kStages * kRows * NV * threads * kBytes; }
  static constexpr int kStep = 32 * kBytes;  // from one vector of a thread to the next
  const RowGroup<VEC, NV, kWarps> &g;
  const T *base;  // a valid address
  uint8_t *slot;  // of this thread in stage 0, row 0
  int pitch;      // bytes of all threads' slots of one row
  struct View {
    const uint8_t *p;
    __device__ __forceinline__ Pairs<VEC> get(int i, bool) const {
      float f[VEC];
      reinterpret_cast<const Elems<T, VEC> *>(p + i * kStep)->get(f);
      return Pairs<VEC>(f);
    }
  };
  __device__ __forceinline__ RowRing(const RowGroup<VEC, NV, kWarps> &group, uint8_t *dyn, const void *any, int)
      : g(group), base(reinterpret_cast<const T *>(any)),
        slot(dyn + (threadIdx.x / 32 * 32 * NV + threadIdx.x % 32) * kBytes), pitch((int)blockDim.x * NV * kBytes) {}
  __device__ __forceinline__ void copy_row(int stage, int n, const T *row, bool live) {
    const T *p = row + g.t0;
    const uint32_t dst = tc::smem_u32(slot + (stage * kRows + n) * pitch);
    g.each(live, [&](int i, auto in) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + i * kStep), "l"(in ? p + i * g.step() : base), "r"(in ? kBytes : 0) : "memory");
    });
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // The oldest of the kStages groups committed last has arrived.
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  }
  __device__ __forceinline__ View view(int stage, int n) const {
    return {slot + (stage * kRows + n) * pitch};
  }
};

// Bytes of the 16-byte words that cover a row that begins anywhere in the first,
// and of the offset of its start (in 16 more).
__host__ __device__ __forceinline__ int span_pitch(int row_bytes) { return (row_bytes + 15) / 16 * 16 + 32; }

// Rows off the 16-byte boundary: the group copies the aligned 16-byte words
// that cover the row (the first may begin before the row, in the same word;
// nothing past its end is read), and each thread reads its values one by one
// from where the row begins in them.  (With an asynchronous copy of its own
// for each value 3003 x 1537 fp32 took 14.0 us forward, so 9.8.)
template <typename T, int NV, bool kWarps, int kRows, int kStages, bool kNamed>
struct RowRing<T, 1, NV, kWarps, kRows, kStages, kNamed> {
  static size_t bytes(int d, int threads, int tpr) {
    return (size_t)kStages * kRows * (threads / tpr) * span_pitch(d * (int)sizeof(T));
  }
  const RowGroup<1, NV, kWarps> &g;
  uint8_t *rows;
  int bytes_, pitch;
  struct View {
    const T *p;
    int step;
    __device__ __forceinline__ Pairs<1> get(int i, bool in) const {
      const float f[1] = {in ? (float)p[i * (kWarps ? 32 : step)] : 0.f};
      return Pairs<1>(f);
    }
  };
  __device__ __forceinline__ RowRing(const RowGroup<1, NV, kWarps> &group, uint8_t *dyn, const void *, int d)
      : g(group), bytes_(d * (int)sizeof(T)), pitch(span_pitch(d * (int)sizeof(T))) {
    rows = dyn + (size_t)group.group * kStages * kRows * pitch;
  }
  __device__ __forceinline__ void copy_row(int stage, int n, const T *row, bool live) {
    if (!live) return;
    uint8_t *to = rows + (stage * kRows + n) * pitch;
    const int lead = (int)(reinterpret_cast<uintptr_t>(row) & 15u), span = lead + bytes_;
    const uint8_t *from = reinterpret_cast<const uint8_t *>(row) - lead;
    if (g.t == 0) *reinterpret_cast<int *>(to + pitch - 16) = lead;
    const uint32_t dst = tc::smem_u32(to);
    auto word = [&](int b, int n) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + b), "l"(from + b), "r"(n) : "memory");
    };
    if (kWarps) {
      // (a warp has as many bytes as its vectors, then one word may be left)
      constexpr int kWords = NV * (int)sizeof(T) / 16;
      const int b0 = (g.t / 32 * kWords * 32 + g.t % 32) * 16;
      if (b0 + kWords * 512 <= span) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) word(b0 + i * 512, 16);
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
          if (b0 + i * 512 < span) word(b0 + i * 512, min(16, span - b0 - i * 512));
      }
      const int last = g.tpr * kWords * 16;
      if (g.t == 0 && last < span) word(last, span - last);
    } else {
      for (int b = g.t * 16; b < span; b += g.tpr * 16) word(b, min(16, span - b));
    }
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (g.tpr <= 32)
      __syncwarp();
    else if (kNamed)
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g.group), "r"(g.tpr) : "memory");
    else
      __syncthreads();
  }
  __device__ __forceinline__ View view(int stage, int n) const {
    const uint8_t *at = rows + (stage * kRows + n) * pitch;
    const int lead = *reinterpret_cast<const int *>(at + pitch - 16);
    return {reinterpret_cast<const T *>(at + lead) + g.t0, g.step()};
  }
};

// Offsets of row r and its successors; r moves on in equal steps.
struct RowCursor {
  RowSet s;
  long long r, off;
  __device__ __forceinline__ RowCursor(const RowSet &set, long long first)
      : s(set), r(first), off(row_offset(set, first)) {}
  __device__ __forceinline__ void advance(long long step) {
    r += step;
    off = s.n0 == 1 ? off + step * s.s1 : row_offset(s, r);
  }
  __device__ __forceinline__ long long at(int k) const {
    return k == 0 ? off : s.n0 == 1 ? off + k * s.s1 : row_offset(s, r + k);
  }
};

// VEC values from packed pairs to the row.
template <typename T, int VEC>
__device__ __forceinline__ void store_pairs(const Pairs<VEC> &p, T *o) {
  float f[VEC];
  p.put(f);
  Elems<T, VEC> e;
  e.set(f);
  e.store(o);
}

template <int VEC>
__device__ __forceinline__ Pairs<VEC> param_pairs(const float *p, int c, float other) {
  float f[VEC];
  load_param<VEC>(p, c, other, f);
  return Pairs<VEC>(f);
}

// R rows at a time by tpr threads (blockDim / tpr such groups in a CTA), NV
// vectors of VEC values a thread and row.  The rows are read from their ring
// slots once and stay in registers between the three uses of them, while the
// next kStages - 1 sets of rows are on their way: loads are in flight all the
// time.  kKeep: the gains and biases of the thread's columns stay in registers
// (from L1 they would be four times the row's own traffic).
// Bound by memory: 16384 x 4096 bf16 42.9 us, 6.3 TB/s; fp32 8192 x 2048 23.8 us,
// 5.6 TB/s.  Value by value (rows off the 16-byte boundary) by the instructions
// a value takes: fp32 8192 x 2047 25.4 us, bf16 8192 x 2047 18.6 us, bf16 8001 x
// 4097 35.3 us.  kWarps: a warp's vectors are
// neighbours; for 16-byte vectors those of the whole group interleave (42.9 us,
// with kWarps 45.8).
template <typename T, int VEC, int NV, int R, int kStages, bool kKeep, int kThreads, bool kWarps>
__global__ void __launch_bounds__(kThreads)
ln_fwd_kernel(const LnArgs a, int tpr) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ __align__(16) float red[2][R][kRed];
  pdl_launch_dependents();
  pdl_wait();
  if (tpr > 32) clear_red(&red[0][0][0], 2 * R * kRed);
  constexpr int NP = Pairs<VEC>::N;
  const RowGroup<VEC, NV, kWarps> g(tpr, a.d);
  const int group = g.group, groups = blockDim.x / tpr;
  const float inv_d = 1.f / (float)a.d;
  float2 wk[kKeep ? NV : 1][NP], bk[kKeep ? NV : 1][NP];
  if (kKeep)
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (g.has(i)) {
        const Pairs<VEC> w = param_pairs<VEC>(a.w, g.t0 + i * g.step(), 1.f);
        const Pairs<VEC> b = param_pairs<VEC>(a.b, g.t0 + i * g.step(), 0.f);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          wk[kKeep ? i : 0][j] = w.v[j];
          bk[kKeep ? i : 0][j] = b.v[j];
        }
      }
  RowRing<T, VEC, NV, kWarps, R, kStages, false> ring(g, dyn, a.x, a.d);
  const long long first = ((long long)blockIdx.x * groups + group) * R;
  const long long stride = (long long)gridDim.x * groups * R;
  const T *x = reinterpret_cast<const T *>(a.x);
  T *y = reinterpret_cast<T *>(a.out) + g.t0;
  RowCursor cx(a.sx, first), cy(a.so, first);
  // Copies the rows at the cursor and moves it on.
  auto ahead = [&](int stage) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool live = cx.r + k < a.rows;
      ring.copy_row(stage, k, live ? x + cx.at(k) : x, live);
    }
    ring.commit();
    cx.advance(stride);
  };
  for (int k = 0; k < kStages - 1; ++k) ahead(k);
  int stage = 0;
  // Every thread of a warp takes part in each row's sums; past the last row
  // it works on zeros and writes nothing.
  for (long long r = first; r - group * R < a.rows; r += stride) {
    // the slot that the previous turn read takes the rows furthest ahead
    ahead(stage == 0 ? kStages - 1 : stage - 1);
    ring.wait();
    float2 v[R][NV][NP];
    float s[R], q[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const auto from = ring.view(stage, k);
      float2 s2 = both(0.f);
      g.each(r + k < a.rows, [&](int i, auto in) {
        const Pairs<VEC> p = from.get(i, in);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          v[k][i][j] = p.v[j];
          s2 = padd<VEC>(s2, p.v[j]);
        }
      });
      s[k] = s2.x + s2.y;
    }
    row_sums<R, false>(s, red[0], tpr);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      s[k] *= inv_d;
      float2 s2 = both(0.f);
      g.each(true, [&](int i, auto in) {
        const float2 nm = both(in ? -s[k] : 0.f);  // zeros past the end stay zeros
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          v[k][i][j] = padd<VEC>(v[k][i][j], nm);
          s2 = pfma<VEC>(v[k][i][j], v[k][i][j], s2);
        }
      });
      q[k] = s2.x + s2.y;
    }
    row_sums<R, false>(q, red[1], tpr);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool live = r + k < a.rows;
      const float rstd = rsqrtf(fmaf(q[k], inv_d, a.eps));
      if (g.t == 0 && live) {
        if (a.mean) a.mean[r + k] = s[k];
        if (a.rstd) a.rstd[r + k] = rstd;
      }
      const float2 rr = both(rstd);
      T *o = y + cy.at(k);
      g.each(live, [&](int i, auto in) {
        if (!in) return;
        const Pairs<VEC> w = kKeep ? Pairs<VEC>() : param_pairs<VEC>(a.w, g.t0 + i * g.step(), 1.f);
        const Pairs<VEC> b = kKeep ? Pairs<VEC>() : param_pairs<VEC>(a.b, g.t0 + i * g.step(), 0.f);
        Pairs<VEC> n;
#pragma unroll
        for (int j = 0; j < NP; ++j)
          n.v[j] = pfma<VEC>(pmul<VEC>(v[k][i][j], rr), kKeep ? wk[kKeep ? i : 0][j] : w.v[j],
                             kKeep ? bk[kKeep ? i : 0][j] : b.v[j]);
        store_pairs<T, VEC>(n, o + i * g.step());
      });
    }
    cy.advance(stride);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
}

// Rows too long for registers: the row is read three times (the second and
// third reading come from the caches), which bounds the kernel by what the L2
// gives: 2048 x 40000 bf16 145 us, 2.3 TB/s of the row's own bytes; fp32 2048 x
// 20000 97 us.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
ln_fwd_long_kernel(const LnArgs a) {
  __shared__ float red[2][1][kRed];
  pdl_launch_dependents();
  pdl_wait();
  clear_red(&red[0][0][0], 2 * kRed);
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
    row_sums<1, false>(s, red[0], blockDim.x);
    const float mean = s[0] * inv_d;
    for (int c = t0; c < a.d; c += step) {
      e.load(x + c);
      e.get(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[0] = fmaf(v[j] - mean, v[j] - mean, q[0]);
    }
    row_sums<1, false>(q, red[1], blockDim.x);
    const float rstd = rsqrtf(fmaf(q[0], inv_d, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
    for (int c = t0; c < a.d; c += step) {
      e.load(x + c);
      e.get(v);
      float w[VEC], b[VEC];
      load_param<VEC>(a.w, c, 1.f, w);
      load_param<VEC>(a.b, c, 0.f, b);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[j] = fmaf((v[j] - mean) * rstd, w[j], b[j]);
      e.set(v);
      e.store(y + c);
    }
  }
}

// dx of the CTA's rows, and the sums of dy h and dy over them: R rows at a
// time by tpr threads, blockDim / tpr such groups in a CTA.  Each thread keeps
// the sums of its own NV x VEC columns in registers for the whole call: that is
// what leaves one CTA of 512 threads an SM, and bounds the kernel by the latency
// of each row's steps at 16 warps rather than by memory (8192 x 4096 bf16: 58% of
// the issue slots, 48% of DRAM; 43 us with the sum over CTAs, 4.7 TB/s; fp32 8192 x
// 2048: 37 us, 5.5 TB/s).  Sums kept in shared memory, or added by atomics, would
// cost each value a read and a write there, and atomics an order that changes.
// The rows come through the ring and are read from it twice, before and after
// the rows' sums.  kKeep: the gains of the thread's columns are in registers
// too.  kHold: h and dy w stay in registers between the two uses instead
// (8192 x 4096 bf16: 45 us one row at a time with it, 44 two rows at a time
// without); values read one by one are held always, since others' copies take
// their place.
template <typename T, int VEC, int NV, int R, int kStages, bool kKeep, int kThreads, bool kHold, bool kWarps>
__global__ void __launch_bounds__(kThreads)
ln_bwd_kernel(const LnArgs a, int tpr, float *__restrict__ part) {
  extern __shared__ __align__(16) uint8_t dyn[];  // ring, then the CTA's sums
  __shared__ __align__(16) float red[2][2 * R][kRed];
  pdl_launch_dependents();
  pdl_wait();
  if (tpr > 32) clear_red(&red[0][0][0], 4 * R * kRed);
  constexpr int NP = Pairs<VEC>::N;
  const RowGroup<VEC, NV, kWarps> grp(tpr, a.d);
  const int group = grp.group, groups = blockDim.x / tpr;
  const float inv_d = 1.f / (float)a.d;
  float2 aw[NV][NP], ab[NV][NP], wk[kKeep ? NV : 1][NP];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) aw[i][j] = ab[i][j] = both(0.f);
  if (kKeep)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pairs<VEC> w;
      if (grp.has(i)) w = param_pairs<VEC>(a.w, grp.t0 + i * grp.step(), 1.f);
#pragma unroll
      for (int j = 0; j < NP; ++j) wk[kKeep ? i : 0][j] = w.v[j];
    }
  RowRing<T, VEC, NV, kWarps, 2 * R, kStages, true> ring(grp, dyn, a.x, a.d);
  const long long first = ((long long)blockIdx.x * groups + group) * R;
  const long long stride = (long long)gridDim.x * groups * R;
  const T *x = reinterpret_cast<const T *>(a.x), *dy = reinterpret_cast<const T *>(a.dy);
  T *dx = reinterpret_cast<T *>(a.out) + grp.t0;
  RowCursor cx(a.sx, first), cg(a.sg, first), co(a.so, first);
  auto ahead = [&](int stage) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const bool live = cx.r + k < a.rows;
      ring.copy_row(stage, 2 * k, live ? x + cx.at(k) : x, live);
      ring.copy_row(stage, 2 * k + 1, live ? dy + cg.at(k) : dy, live);
    }
    ring.commit();
    cx.advance(stride);
    cg.advance(stride);
  };
  for (int k = 0; k < kStages - 1; ++k) ahead(k);
  float mean_n[R], rstd_n[R];  // of the next rows
  auto stats = [&](long long r) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean_n[k] = r + k < a.rows ? a.mean[r + k] : 0.f;
      rstd_n[k] = r + k < a.rows ? a.rstd[r + k] : 0.f;
    }
  };
  stats(first);
  int par = 0, stage = 0;
  // As in the forward, threads past the last row work on zeros.
  for (long long r = first; r - group * R < a.rows; r += stride, par ^= 1) {
    float2 nm[R], rr[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      nm[k] = both(-mean_n[k]);
      rr[k] = both(rstd_n[k]);
    }
    stats(r + stride);
    // the slot that the previous turn read takes the rows furthest ahead
    ahead(stage == 0 ? kStages - 1 : stage - 1);
    ring.wait();
    float s[2 * R];
    float2 hk[kHold ? R : 1][kHold ? NV : 1][NP], gk[kHold ? R : 1][kHold ? NV : 1][NP];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const auto fx = ring.view(stage, 2 * k), fg = ring.view(stage, 2 * k + 1);
      float2 s0 = both(0.f), s1 = both(0.f);
      grp.each(r + k < a.rows, [&](int i, auto in) {
        const Pairs<VEC> px = fx.get(i, in), g = fg.get(i, in);
        Pairs<VEC> w;
        if (!kKeep && in) w = param_pairs<VEC>(a.w, grp.t0 + i * grp.step(), 1.f);
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float2 h = pmul<VEC>(padd<VEC>(px.v[j], nm[k]), rr[k]);
          aw[i][j] = pfma<VEC>(g.v[j], h, aw[i][j]);
          ab[i][j] = padd<VEC>(ab[i][j], g.v[j]);
          const float2 gw = pmul<VEC>(g.v[j], kKeep ? wk[kKeep ? i : 0][j] : w.v[j]);
          s0 = padd<VEC>(s0, gw);
          s1 = pfma<VEC>(gw, h, s1);
          if (kHold) {
            hk[kHold ? k : 0][kHold ? i : 0][j] = h;
            gk[kHold ? k : 0][kHold ? i : 0][j] = gw;
          }
        }
      });
      s[2 * k] = s0.x + s0.y;
      s[2 * k + 1] = s1.x + s1.y;
    }
    row_sums<2 * R, true>(s, red[par], tpr);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      // dx = rstd (g - c1 - h c2)
      const float2 c1 = both(-s[2 * k] * inv_d), c2 = both(-s[2 * k + 1] * inv_d);
      const float2 rc2 = both(__fmul_rn(rr[k].x, c2.x));  // h c2 = (x - mean) rstd c2
      const bool live = r + k < a.rows;
      T *o = dx + co.at(k);
      const auto fx = ring.view(stage, 2 * k), fg = ring.view(stage, 2 * k + 1);
      grp.each(live, [&](int i, auto in) {
        if (!in) return;
        Pairs<VEC> g;
        if (kHold) {
#pragma unroll
          for (int j = 0; j < NP; ++j)
            g.v[j] = pmul<VEC>(rr[k], padd<VEC>(gk[kHold ? k : 0][kHold ? i : 0][j], pfma<VEC>(hk[kHold ? k : 0][kHold ? i : 0][j], c2, c1)));
        } else {
          const Pairs<VEC> px = fx.get(i, true);
          const Pairs<VEC> w = kKeep ? Pairs<VEC>() : param_pairs<VEC>(a.w, grp.t0 + i * grp.step(), 1.f);
          g = fg.get(i, true);
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const float2 gw = pmul<VEC>(g.v[j], kKeep ? wk[kKeep ? i : 0][j] : w.v[j]);
            g.v[j] = pmul<VEC>(rr[k], padd<VEC>(gw, pfma<VEC>(padd<VEC>(px.v[j], nm[k]), rc2, c1)));
          }
        }
        store_pairs<T, VEC>(g, o + i * grp.step());
      });
    }
    co.advance(stride);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  if (!part) return;
  // The sums of each warp (rows of fewer than 32 threads) or row group go to
  // shared memory; the CTA adds them in order.
  for (int k = tpr; k < 32; k <<= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        aw[i][j].x += __shfl_xor_sync(0xffffffffu, aw[i][j].x, k);
        ab[i][j].x += __shfl_xor_sync(0xffffffffu, ab[i][j].x, k);
        aw[i][j].y += __shfl_xor_sync(0xffffffffu, aw[i][j].y, k);
        ab[i][j].y += __shfl_xor_sync(0xffffffffu, ab[i][j].y, k);
      }
  const int unit_threads = tpr < 32 ? 32 : tpr, units = blockDim.x / unit_threads;
  float *out = part + (size_t)blockIdx.x * 2 * a.d, *sums = reinterpret_cast<float *>(dyn);
  float *mine = units > 1 ? sums + (size_t)(threadIdx.x / unit_threads) * 2 * a.d : out;
  asm volatile("cp.async.wait_all;" ::: "memory");  // zeros for rows past the last one
  __syncthreads();  // every copy to the ring has been read
  if (tpr >= 32 || (int)(threadIdx.x & 31) < tpr)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = grp.t0 + i * grp.step();
      if (grp.has(i))
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          mine[c + 2 * j] = aw[i][j].x;
          mine[a.d + c + 2 * j] = ab[i][j].x;
          if (VEC > 1) {
            mine[c + 2 * j + 1] = aw[i][j].y;
            mine[a.d + c + 2 * j + 1] = ab[i][j].y;
          }
        }
    }
  if (units == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) {
    float v = sums[c];
    for (int k = 1; k < units; ++k) v += sums[(size_t)k * 2 * a.d + c];
    out[c] = v;
  }
}

// Rows too long for one CTA's registers, in two passes: mean(g) and
// mean(g h) of each row (stat[r][2]), then dx and the column sums by column
// blocks.  x and dy are read twice, 5 row elements a value instead of 3: 2048 x
// 40000 bf16 174 us, 4.7 TB/s for what it moves; fp32 2048 x 16384 115 us.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
ln_bwd_stat_kernel(const LnArgs a, float *__restrict__ stat) {
  __shared__ float red[2][2][kRed];
  pdl_launch_dependents();
  pdl_wait();
  clear_red(&red[0][0][0], 4 * kRed);
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
      float w[VEC];
      load_param<VEC>(a.w, c, 1.f, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        g[j] *= w[j];
        s[0] += g[j];
        s[1] = fmaf(g[j], (h[j] - mean) * rstd, s[1]);
      }
    }
    row_sums<2, false>(s, red[par], blockDim.x);
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
  for (int j = 0; j < VEC; ++j) aw[j] = ab[j] = 0.f;
  load_param<VEC>(a.w, c, 1.f, w);
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
// not depend on which CTA finished first.  A CTA has 32 columns and a warp for
// every 32nd partial row, so that at most five loads follow one another: 152 x
// 2 x 4096 values, 5 MB, take 6 us alone and cold, nearly all of it latency.
// (CTAs of 256 threads were no faster.)
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

// 16-byte vectors need every row of every operand on a 16-byte boundary.
bool rows_aligned(const void *p, const RowSet &s, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (s.n1 == 1 || s.s1 * esz % 16 == 0) &&
         (s.n0 == 1 || s.s0 * esz % 16 == 0);
}

bool param_aligned(const float *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Threads a row for n vectors with at most `most` a thread: lanes of a warp
// (a power of two) or whole warps.
int threads_per_row(int n, int most) {
  const int t = (n + most - 1) / most;
  if (t > 16) return (t + 31) / 32 * 32;
  int p = 1;
  while (p < t) p *= 2;
  return p;
}

// One `done` word per kernel: kKern is part of the type.
template <auto kKern, typename... Args>
cudaError_t launch_with(int grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  static std::atomic<unsigned> done{0};
  if (smem > 32 * 1024) {
    const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kKern), done);
    if (e != cudaSuccess) return e;
  }
  return launch_k(kKern, dim3(grid), dim3(threads), smem, st, true, args...);
}

template <typename T, int VEC, int NV, int R, int kStages, bool kKeep, int kThreads>
cudaError_t fwd(const LnArgs &a, int tpr, int per_sm, cudaStream_t st) {
  const int threads = tpr > 32 ? tpr : 128, rows = threads / tpr * R;
  const size_t smem = RowRing<T, VEC, NV, true, R, kStages, false>::bytes(a.d, threads, tpr);
  // CTAs that stay for the whole call, per_sm threads an SM, less where the
  // rings fill its shared memory.
  const long long fit = std::max<long long>(1, std::min<long long>(per_sm / threads, 220 * 1024 / (smem + 1024)));
  const long long want = (a.rows + rows - 1) / rows, most = device_sms() * fit;
  const int grid = (int)std::min(want, most);
  // (values one by one in whole warps: kWarps; below 32 threads no wide rows)
  if constexpr (VEC == 1)
    if (tpr >= 32)
      return launch_with<ln_fwd_kernel<T, VEC, NV, R, kStages, kKeep, kThreads, true>>(grid, threads, smem, st, a, tpr);
  if constexpr (VEC > 1 || NV == 8 || R == 2)
    return launch_with<ln_fwd_kernel<T, VEC, NV, R, kStages, kKeep, kThreads, false>>(grid, threads, smem, st, a, tpr);
  return cudaErrorInvalidValue;
}

template <typename T, int VEC>
cudaError_t fwd_any(const LnArgs &a, cudaStream_t st) {
  const int n = (a.d + VEC - 1) / VEC;
  const int t8 = threads_per_row(n, 8 / VEC), t16 = threads_per_row(n, 16 / VEC), t32 = threads_per_row(n, 32 / VEC);
  // Few rows: 8 values a thread while that leaves the SMs with at most 1024
  // threads each.
  if (t8 <= 1024 && a.rows * t8 <= (long long)device_sms() * 1024)
    return fwd<T, VEC, 8 / VEC, 1, 2, false, 1024>(a, t8, 1024, st);
  // Short rows off the 16-byte boundary: one row of 8 (65536 rows, bf16: d = 31
  // 7.3 us, two rows of 16 13.3; d = 255 24.4 and 26.7; d = 127 18.7 and 16.7).
  if constexpr (VEC == 1)
    if (t8 == 32 || t8 <= 8) return fwd<T, VEC, 8, 1, 3, true, 1024>(a, t8, 1536, st);
  // Else two rows of 16 values a thread or one of 32, gains and biases in
  // registers either way.  Rows of 32: above 4096 values (8192 rows, bf16: d =
  // 5120 28.0 us, two of 16 40.3; 8192 43.8 and 48.3; 4096 x 16384 46.0; at 4096
  // two of 16 are better, 42.9 and 46.8 for 16384 rows), and for bf16 off the
  // 16-byte boundary where no more than an eighth more places stay empty (8192 x
  // 3001 24.2 and 27.8; 8001 x 4097 35.3 and 51.7; not 8192 x 1535, 16.8 and 15.4).
  const bool one = a.d > 4096 || (VEC == 1 && sizeof(T) == 2 && t32 >= 32 && t32 * 16 <= t16 * 9);
  constexpr int kStages = sizeof(T) == 4 ? 2 : 3;
  if (one && t32 <= 512) return fwd<T, VEC, 32 / VEC, 1, kStages, true, 512>(a, t32, 512, st);
  if (t16 <= 512) return fwd<T, VEC, 16 / VEC, 2, kStages, true, 512>(a, t16, 512, st);
  if constexpr (VEC == 8)
    if (t32 <= 1024) return fwd<T, 8, 4, 1, 2, false, 1024>(a, t32, 1024, st);
  const long long cap = 1LL << 30;
  return launch_k(ln_fwd_long_kernel<T, VEC>, dim3((unsigned)(a.rows < cap ? a.rows : cap)),
                  dim3(1024), 0, st, true, a);
}

constexpr int kBwdStages = 3;

template <typename T, int VEC, int NV, int R, int kStages, bool kKeep, int kThreads, bool kHold>
cudaError_t bwd(const LnArgs &a, const LnBwdPlan &pl, float *part, cudaStream_t st) {
  const int units = pl.threads / std::max(pl.tpr, 32);
  const size_t smem = std::max(units > 1 ? (size_t)units * 2 * a.d * sizeof(float) : 0,
                               RowRing<T, VEC, NV, true, 2 * R, kStages, true>::bytes(a.d, pl.threads, pl.tpr));
  if constexpr (NV * VEC < 32)  // (32 values a thread: wide rows only)
    if (pl.tpr < 32 || VEC > 1)
      return launch_with<ln_bwd_kernel<T, VEC, NV, R, kStages, kKeep, kThreads, kHold, false>>(
          pl.groups, pl.threads, smem, st, a, pl.tpr, part);
  return launch_with<ln_bwd_kernel<T, VEC, NV, R, kStages, kKeep, kThreads, kHold, true>>(
      pl.groups, pl.threads, smem, st, a, pl.tpr, part);
}

template <typename T, int VEC>
cudaError_t bwd_any(const LnArgs &a, const LnBwdPlan &pl, const float *stat, float *part,
                    cudaStream_t st) {
  if (pl.two_pass) {
    const int cols = 256 * VEC;
    return launch_k(ln_bwd_cols_kernel<T, VEC>, dim3((a.d + cols - 1) / cols, pl.groups), dim3(256),
                    0, st, true, a, stat, part);
  }
  if constexpr (VEC == 8)
    // (two stages: three would leave L1 no room for the gains; 4096 x 16384 118 us and 134)
    if (pl.wide) return bwd<T, 8, 4, 1, 2, false, 512, false>(a, pl, part, st);
  if constexpr (VEC == 1)
    if (pl.narrow) return bwd<T, 1, 8, 1, kBwdStages, true, 512, true>(a, pl, part, st);
  return bwd<T, VEC, 16 / VEC, VEC == 8 ? 2 : 1, kBwdStages, true, 512, VEC == 1>(a, pl, part, st);
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
  const bool v = a.d % vec == 0 && rows_aligned(a.x, a.sx, esz) && rows_aligned(a.out, a.so, esz) &&
                 param_aligned(a.w) && param_aligned(a.b);
  if (bf16) return v ? fwd_any<__nv_bfloat16, 8>(a, st) : fwd_any<__nv_bfloat16, 1>(a, st);
  return v ? fwd_any<float, 4>(a, st) : fwd_any<float, 1>(a, st);
}

LnBwdPlan layernorm_bwd_plan(const LnArgs &a, int bf16) {
  LnBwdPlan pl;
  const int esz = bf16 ? 2 : 4, vec = 16 / esz;
  pl.vec = a.d % vec == 0 && rows_aligned(a.x, a.sx, esz) && rows_aligned(a.dy, a.sg, esz) &&
           rows_aligned(a.out, a.so, esz) && param_aligned(a.w);
  // Columns a thread: 16 (up to 256 values off the 16-byte boundary 8: 65536 x
  // 31 bf16 12.2 us, with 16 17.5), above 8192 columns 32 (bf16), else two passes.
  const int V = pl.vec ? vec : 1, n = (a.d + V - 1) / V;
  pl.narrow = !pl.vec && a.d <= 256;
  pl.tpr = threads_per_row(n, pl.narrow ? 8 : 16 / V);
  if (pl.tpr > 512) {
    pl.wide = V == 8 && pl.tpr <= 1024;
    pl.two_pass = !pl.wide;
    pl.tpr = threads_per_row(n, 32 / V);
  }
  if (pl.two_pass) {
    pl.groups = (int)std::min<long long>(a.rows, kTwoPassGroups);
    return pl;
  }
  // One CTA of up to 512 threads an SM: as many row groups as fit, for few
  // rows no more than share out over all SMs.  (At most 15 groups of several
  // warps: each has a named barrier.)
  const long long sms = device_sms(), R = V == 8 && !pl.wide ? 2 : 1;
  const int most = 512;
  long long fit = pl.tpr > 32 ? std::min(most / pl.tpr, 15) : most / pl.tpr;
  if (!pl.vec) {  // (short rows: no more than 192 KB of them, in whole warps)
    fit = std::min<long long>(fit, 192 * 1024 / (kBwdStages * 2 * span_pitch(a.d * esz)));
    if (pl.tpr < 32) fit = fit * pl.tpr / 32 * 32 / pl.tpr;
    fit = std::max<long long>(fit, 1);
  }
  long long at_once = std::min(fit, std::max<long long>(1, a.rows / (sms * R)));
  while (pl.tpr < 32 && at_once * pl.tpr % 32) ++at_once;
  pl.threads = (int)at_once * pl.tpr;
  pl.groups = (int)std::min((a.rows + at_once * R - 1) / (at_once * R), sms);
  return pl;
}

size_t layernorm_bwd_bytes(long long rows, int d) {
  const long long most = std::max(device_sms(), kTwoPassGroups);
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
