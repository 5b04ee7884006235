// The short causal convolution of each channel over its sequence,
//   pre_t = b + sum_k w_k x_{t-W+1+k},   y_t = silu(pre_t)  (or pre_t),
// where the W - 1 inputs before the first token are a kept state (or 0), and
// its gradients: with d_t = dy_t silu'(pre_t),
//   dx_t = sum_k w_k d_{t+W-1-k},   dw_k = sum_t d_t x_{t-W+1+k},   db = sum_t d_t.
// fp32 arithmetic.  Bound by memory: two (forward) or three row elements a
// value.  A thread walks a run of tokens of its channels with the last W
// inputs in registers, so that each input is read once, but for the W - 1
// tokens at the ends of a run.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "scan.cuh"

namespace ret {

namespace {

using namespace scan;

constexpr int kThreads = 256;

// V neighbouring channels as they were read: 4, 2 or 1.
template <typename T, int V>
struct __align__(V * sizeof(T)) Chans {
  T v[V];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (V == 1)
      v[0] = *p;
    else if constexpr (V * sizeof(T) == 4)
      *reinterpret_cast<uint32_t *>(v) = *reinterpret_cast<const uint32_t *>(p);
    else if constexpr (V * sizeof(T) == 8)
      *reinterpret_cast<uint2 *>(v) = *reinterpret_cast<const uint2 *>(p);
    else
      *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = from_float<T>(0.f);
  }
  __device__ __forceinline__ float get(int i) const { return to_float(v[i]); }
  __device__ __forceinline__ static void store(T *p, const float (&f)[V]) {
    if constexpr (V == 1)
      *p = from_float<T>(f[0]);
    else if constexpr (V == 2)
      store_two<T, true>(p, 2, f[0], f[1]);
    else
      store_four<T, true>(p, 4, f);
  }
};

// c + a b, a b and the sigmoid for V channels, on packed pairs.
template <int V>
__device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], float (&c)[V]) {
  if constexpr (V == 1) {
    c[0] = fmaf(a[0], b[0], c[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = tc::fma2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
      c[i] = r.x;
      c[i + 1] = r.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void mul_v(const float (&a)[V], const float (&b)[V], float (&c)[V]) {
  if constexpr (V == 1) {
    c[0] = a[0] * b[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = tc::mul2(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      c[i] = r.x;
      c[i + 1] = r.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void sigmoid_v(const float (&a)[V], float (&c)[V]) {
  if constexpr (V == 1) {
    c[0] = sigmoid(a[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 r = sigmoid2(make_float2(a[i], a[i + 1]));
      c[i] = r.x;
      c[i + 1] = r.y;
    }
  }
}

__device__ __forceinline__ int conv_tokens(const ConvArgs &a, int b) {
  if (!a.lengths) return a.N;
  const long long n = a.len64 ? reinterpret_cast<const long long *>(a.lengths)[b]
                              : (long long)reinterpret_cast<const int *>(a.lengths)[b];
  return (int)(n < 0 ? 0 : n > a.N ? a.N : n);
}

// The taps of V channels (V W neighbouring values) and their biases.
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int e, bool vec, float (&w)[W][V], float (&bias)[V]) {
  float f[V * W];
  const float *p = a.w + (size_t)e * W;
  if (V * W % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 3 < V * W; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(p + i);
      f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V * W; ++i) f[i] = p[i];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.b ? a.b[e + v] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][v] = f[v * W + k];
  }
}

// The input at position t >= -(W - 1) of a sequence: of the state before 0.
template <typename T, int V, int W>
__device__ __forceinline__ Chans<T, V> input_at(const ConvArgs &a, int b, int e, int t) {
  Chans<T, V> c;
  if (t >= 0)
    c.load(reinterpret_cast<const T *>(a.x) + b * a.sx[0] + t * a.sx[1] + e);
  else if (a.state_in)
    c.load(reinterpret_cast<const T *>(a.state_in) + ((size_t)b * (W - 1) + (W - 1 + t)) * a.E + e);
  else
    c.zero();
  return c;
}

// run: tokens of a thread, at least W - 1 (then only the first run reads the
// state, which state_out may be).  U tokens' loads (64 bytes) are in flight; the inputs
// stay as they were read until their turn (8192 x 4096 bf16 32 us, 4.2 TB/s: the
// loads' latency at 24 warps an SM, 2.6 of 8.8 cycles between a warp's
// instructions, and their issue, 52% of the slots; with four tokens of eight
// channels in flight, converted at once, 124; through shared memory 44 for 37).  fp32
// 54 us for 2 x 4096 x 4096; its window and loads pass 80 registers with four taps
// (100 bytes spilled).
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads, 3)
conv_fwd_kernel(const ConvArgs a, int run, int runs, int vec_taps) {
  constexpr int U = V * sizeof(T) == 16 ? 4 : 8;
  pdl_launch_dependents();
  pdl_wait();
  const int nv = a.E / V, b = blockIdx.y;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nv * runs) return;
  const int r = (int)(i / nv), e = (int)(i - (long long)r * nv) * V;
  const int n = conv_tokens(a, b), t0 = r * run, t1 = min(a.N, t0 + run), live = min(n, t1);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + e;
  T *y = reinterpret_cast<T *>(a.out) + b * a.so[0] + e;
  Chans<T, V> in[U];
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (t0 + j < live) in[j].load(x + (t0 + j) * a.sx[1]);
  float w[W][V], bias[V], win[W][V];  // win[k]: the input W - 1 - k tokens before
  if (t0 < live) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const Chans<T, V> c = input_at<T, V, W>(a, b, e, t0 - (W - 1) + k);
#pragma unroll
      for (int v = 0; v < V; ++v) win[k + 1][v] = c.get(v);
    }
    load_taps<V, W>(a, e, vec_taps, w, bias);
  }
  auto step = [&](int j, int t, bool more) {
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
      win[W - 1][v] = in[j].get(v);
      o[v] = bias[v];
    }
#pragma unroll
    for (int k = 0; k < W; ++k) fma_v<V>(w[k], win[k], o);
    if (a.silu) {
      float sg[V];
      sigmoid_v<V>(o, sg);
      mul_v<V>(o, sg, o);
    }
    if (more) in[j].load(x + (t + U) * a.sx[1]);
    Chans<T, V>::store(y + t * a.so[1], o);
  };
  int t = t0;
  for (; t + 2 * U <= live; t += U)
#pragma unroll
    for (int j = 0; j < U; ++j) step(j, t + j, true);
  for (; t < live; t += U)
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (t + j < live) step(j, t + j, t + j + U < live);
  const float zero[V] = {};
  for (t = max(t0, live); t < t1; ++t) Chans<T, V>::store(y + t * a.so[1], zero);
  if (r == 0 && a.state_out) {
    Chans<T, V> s[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) s[k] = input_at<T, V, W>(a, b, e, n - (W - 1) + k);
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      float f[V];
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = s[k].get(v);
      Chans<T, V>::store(reinterpret_cast<T *>(a.state_out) + ((size_t)b * (W - 1) + k) * a.E + e, f);
    }
  }
}

// A thread's tokens on their way, n tensors' values each: in shared memory, where a
// thread reads what it copied itself (no barrier), U tokens at a time, kAhead
// such steps ahead of their use; bf16 values one by one wait in registers.
template <typename T, int V, int U, int n>
struct Ahead {
  static constexpr bool kCopies = V * sizeof(T) >= 4;
  static constexpr int kAhead = kCopies ? 4 : 1, kSlots = kCopies ? kAhead * U : 0;
  static constexpr size_t kBytes = (size_t)kSlots * n * kThreads * sizeof(Chans<T, V>);
  Chans<T, V> *ring;
  Chans<T, V> now[U][n];  // (registers, or what take() read)
  __device__ __forceinline__ Ahead(uint8_t *dyn) : ring(reinterpret_cast<Chans<T, V> *>(dyn) + threadIdx.x) {}
  // Token j of step s from p[0 .. n), where it is there.
  __device__ __forceinline__ void fetch(int s, int j, bool there, const T *const (&p)[n]) {
    if constexpr (kCopies) {
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (there)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(ring + (((s % kAhead) * U + j) * n + i) * kThreads)),
                       "l"(p[i]), "n"((int)(V * sizeof(T)))
                       : "memory");
    } else if (there) {
#pragma unroll
      for (int i = 0; i < n; ++i) now[j][i].load(p[i]);
    }
  }
  __device__ __forceinline__ void commit() {
    if (kCopies) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Step s has arrived (kAhead - 1 younger ones may be on their way).
  __device__ __forceinline__ void take(int s) {
    if constexpr (kCopies) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < n; ++i) now[j][i] = ring[(((s % kAhead) * U + j) * n + i) * kThreads];
    }
  }
};

template <typename T, int V>
constexpr int kBwdStep = V * sizeof(T) >= 4 ? 4 : 8;  // (in registers: what a step loads is all that is on its way)

// The taps, the window, the gradients' window and the sums of a thread's channels
// take most of its registers: four channels (bf16) leave two CTAs an SM, two three.
// 2 x 4096 x 4096 bf16 60 us (3.3 TB/s): a token's chain of arithmetic at 16 warps an
// SM (56% of the issue slots, stalls of fixed latency and of the packed pipe before
// those of loads; four taps spill 22 bytes); with two channels a thread 70, with
// four whose tokens waited in registers 222 (one CTA an SM).  fp32 85 us.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads, V == 4 ? 2 : 3)
conv_bwd_kernel(const ConvArgs a, int run, int runs, int vec_taps, float *__restrict__ part) {
  constexpr int U = kBwdStep<T, V>;
  using In = Ahead<T, V, U, 2>;
  extern __shared__ __align__(16) uint8_t dyn[];
  pdl_launch_dependents();
  pdl_wait();
  const int nv = a.E / V, b = blockIdx.y;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nv * runs) return;
  const int r = (int)(i / nv), e = (int)(i - (long long)r * nv) * V;
  const int n = conv_tokens(a, b), t0 = r * run, t1 = min(a.N, t0 + run);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + e;
  const T *dy = reinterpret_cast<const T *>(a.dy) + b * a.sg[0] + e;
  T *dx = reinterpret_cast<T *>(a.out) + b * a.so[0] + e;
  const int last = t1 + W - 1, there = min(n, last);  // tokens walked, of them the sequence's
  In in(dyn);
  auto fetch = [&](int s) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int t = t0 + s * U + j;
      const T *const p[2] = {x + t * a.sx[1], dy + t * a.sg[1]};
      in.fetch(s, j, t < there, p);
    }
    in.commit();
  };
  if (In::kCopies)
    for (int s = 0; s < In::kAhead; ++s) fetch(s);
  float w[W][V], bias[V], win[W][V], d[W][V], dw[W][V], db[V];  // d[k]: of the token k before
  load_taps<V, W>(a, e, vec_taps, w, bias);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) win[k][v] = d[k][v] = dw[k][v] = 0.f;
  }
  if (t0 < n)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const Chans<T, V> c = input_at<T, V, W>(a, b, e, t0 - (W - 1) + k);
#pragma unroll
      for (int v = 0; v < V; ++v) win[k + 1][v] = c.get(v);
    }
  // Token at's d, and with it dx of token at - (W - 1).  kInner: a token of the run
  // and the sequence whose dx is the run's too, and no state behind it.
  auto step = [&](int j, int at, auto inner) {
    constexpr bool kInner = decltype(inner)::value;
    const int o = at - (W - 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int k = W - 1; k > 0; --k) d[k][v] = d[k - 1][v];
    if (kInner || at < there) {
      const bool mine = kInner || at < t1;  // (what lies behind the run belongs to the next one's sums)
      float pre[V], dv[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
        win[W - 1][v] = in.now[j][0].get(v);
        dv[v] = in.now[j][1].get(v);
        pre[v] = bias[v];
      }
      if (a.silu) {  // dy sg (1 + pre (1 - sg))
        float sg[V], t[V];
#pragma unroll
        for (int k = 0; k < W; ++k) fma_v<V>(w[k], win[k], pre);
        sigmoid_v<V>(pre, sg);
#pragma unroll
        for (int v = 0; v < V; ++v) t[v] = 1.f - sg[v];
        mul_v<V>(dv, sg, dv);
        mul_v<V>(pre, t, t);
        fma_v<V>(dv, t, dv);
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        d[0][v] = dv[v];
        if (mine) db[v] += dv[v];
      }
      if (mine)
#pragma unroll
        for (int k = 0; k < W; ++k) fma_v<V>(dv, win[k], dw[k]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) d[0][v] = 0.f;
    }
    if (kInner || o >= t0 || (r == 0 && o < 0)) {
      float out[V];
      mul_v<V>(w[0], d[0], out);
#pragma unroll
      for (int k = 1; k < W; ++k) fma_v<V>(w[k], d[k], out);
      // what the state after the sequence passes back to the last W - 1 inputs
      const int m = o - (n - (W - 1));
      if (!kInner && a.dstate_out && m >= 0 && m < W - 1) {
        Chans<T, V> s;
        s.load(reinterpret_cast<const T *>(a.dstate_out) + ((size_t)b * (W - 1) + m) * a.E + e);
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] += s.get(v);
      }
      if (kInner || o >= 0)
        Chans<T, V>::store(dx + o * a.so[1], out);
      else if (a.dstate_in)
        Chans<T, V>::store(reinterpret_cast<T *>(a.dstate_in) + ((size_t)b * (W - 1) + W - 1 + o) * a.E + e, out);
    }
  };
  for (int t = t0, s = 0; t < last; t += U, ++s) {
    if (!In::kCopies) fetch(s);
    in.take(s);
    if (In::kCopies) fetch(s + In::kAhead);  // (take() has read this step's slots)
    if (t > t0 && t + U <= min(there, t1)) {
#pragma unroll
      for (int j = 0; j < U; ++j) step(j, t + j, std::true_type());
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (t + j < last) step(j, t + j, std::false_type());
    }
  }
  if (!part) return;
  const size_t row = (size_t)b * runs + r, rows = (size_t)a.B * runs;
  float *pb = part + rows * a.E * W + row * a.E + e, *pw = part + (row * a.E + e) * W;
  float f[V * W];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < W; ++k) f[v * W + k] = dw[k][v];
  if constexpr (V >= 2) {  // (E is even, the workspace aligned)
#pragma unroll
    for (int v = 0; v < V; v += 2) *reinterpret_cast<float2 *>(pb + v) = make_float2(db[v], db[v + 1]);
#pragma unroll
    for (int v = 0; v < V * W; v += 2) *reinterpret_cast<float2 *>(pw + v) = make_float2(f[v], f[v + 1]);
  } else {
    pb[0] = db[0];
#pragma unroll
    for (int v = 0; v < W; ++v) pw[v] = f[v];
  }
}

bool aligned(const void *p, const long long s[2], int B, int N, int bytes, int esz) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (N <= 1 || s[1] * esz % bytes == 0) &&
         (B <= 1 || s[0] * esz % bytes == 0);
}

// Tokens of a thread, so that the waves of CTAs (per_sm at once) that the call
// takes are as short as they can be: `ends` more tokens' time go into a run's
// ends (the W - 1 tokens read twice, taps, sums).  8192 x 4096 bf16 forward 32 us,
// with 32 tokens (2.2 waves) 37.
int run_of(const ConvArgs &a, int nv, int per_sm, int ends, int most) {
  const long long slots = (long long)device_sms() * per_sm;
  int best = 4;
  long long least = -1;
  for (int run = 4; run <= most; run += 4) {
    const long long runs = std::max(1, (a.N + run - 1) / run);
    const long long ctas = ((long long)nv * runs + kThreads - 1) / kThreads * std::max(a.B, 1);
    const long long time = (ctas + slots - 1) / slots * (run + ends);
    if (least < 0 || time <= least) {
      least = time;
      best = run;
    }
    if (run >= a.N) break;
  }
  return best;
}
int taps_on(const ConvArgs &a) { return reinterpret_cast<uintptr_t>(a.w) % 16 == 0; }
int runs_of(int N, int run) { return std::max(1, (N + run - 1) / run); }

template <typename T, int V, int W>
cudaError_t fwd(const ConvArgs &a, cudaStream_t st) {
  const int nv = a.E / V, run = run_of(a, nv, 3, 8, 128), runs = runs_of(a.N, run);
  const dim3 grid((unsigned)(((long long)nv * runs + kThreads - 1) / kThreads), a.B);
  return launch_k(conv_fwd_kernel<T, V, W>, grid, dim3(kThreads), 0, st, true, a, run, runs, taps_on(a));
}

template <typename T, int V, int W>
cudaError_t bwd(const ConvArgs &a, float *part, cudaStream_t st) {
  const int runs = conv_bwd_runs(a) / a.B, run = std::max(4, (a.N + runs - 1) / runs);
  const dim3 grid((unsigned)(((long long)(a.E / V) * runs + kThreads - 1) / kThreads), a.B);
  static std::atomic<unsigned> done{0};
  const cudaError_t err = allow_big_smem(reinterpret_cast<const void *>(conv_bwd_kernel<T, V, W>), done);
  if (err != cudaSuccess) return err;
  return launch_k(conv_bwd_kernel<T, V, W>, grid, dim3(kThreads), Ahead<T, V, kBwdStep<T, V>, 2>::kBytes, st, true, a, run, runs, taps_on(a), part);
}

template <typename T, int V>
cudaError_t fwd_taps(const ConvArgs &a, cudaStream_t st) {
  return a.W == 2 ? fwd<T, V, 2>(a, st) : a.W == 3 ? fwd<T, V, 3>(a, st) : fwd<T, V, 4>(a, st);
}

template <typename T, int V>
cudaError_t bwd_taps(const ConvArgs &a, float *part, cudaStream_t st) {
  return a.W == 2 ? bwd<T, V, 2>(a, part, st) : a.W == 3 ? bwd<T, V, 3>(a, part, st) : bwd<T, V, 4>(a, part, st);
}

}  // namespace

// V channels at a time where every row begins on their boundary.
static bool vectors(const ConvArgs &a, int V, const void *const *flat, int n, int esz) {
  const int by = V * esz;
  for (int i = 0; i < n; ++i)
    if (reinterpret_cast<uintptr_t>(flat[i]) % by) return false;
  return a.E % V == 0 && aligned(a.x, a.sx, a.B, a.N, by, esz) && aligned(a.out, a.so, a.B, a.N, by, esz);
}

cudaError_t launch_conv_fwd(const ConvArgs &a, int bf16, cudaStream_t st) {
  const void *flat[] = {a.state_in, a.state_out};
  const bool v = vectors(a, 4, flat, 2, bf16 ? 2 : 4);
  if (bf16) return v ? fwd_taps<__nv_bfloat16, 4>(a, st) : fwd_taps<__nv_bfloat16, 1>(a, st);
  return v ? fwd_taps<float, 4>(a, st) : fwd_taps<float, 1>(a, st);
}

// Runs of tokens over all sequences: those that suit the aligned bf16 form (four
// channels a thread, two CTAs an SM), for every form, since the workspace is sized
// before the tensors' addresses are known.
int conv_bwd_runs(const ConvArgs &a) {
  return runs_of(a.N, run_of(a, std::max(1, a.E / 4), 2, 16, 128)) * a.B;
}

cudaError_t launch_conv_bwd(const ConvArgs &a, int bf16, float *part, cudaStream_t st) {
  const int esz = bf16 ? 2 : 4;
  const void *flat[] = {a.state_in, a.dstate_in, a.dstate_out};
  auto on = [&](int V) { return vectors(a, V, flat, 3, esz) && aligned(a.dy, a.sg, a.B, a.N, V * esz, esz); };
  if (!bf16) return on(2) ? bwd_taps<float, 2>(a, part, st) : bwd_taps<float, 1>(a, part, st);
  if (on(4)) return bwd_taps<__nv_bfloat16, 4>(a, part, st);
  return on(2) ? bwd_taps<__nv_bfloat16, 2>(a, part, st) : bwd_taps<__nv_bfloat16, 1>(a, part, st);
}

}  // namespace ret
