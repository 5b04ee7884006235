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

#include "launch.h"
#include "scan.cuh"

namespace ret {

namespace {

using namespace scan;

constexpr int kThreads = 256;

// V neighbouring channels (16 bytes, 8 bytes or one value).
template <typename T, int V>
struct Chans {
  __device__ __forceinline__ static void load(const T *p, float (&f)[V]) {
    if constexpr (V == 1) {
      f[0] = to_float(*p);
    } else if constexpr (sizeof(T) * V == 16) {
      Elems<T, V> e;
      e.load(p);
      e.get(f);
    } else {
      const uint2 r = *reinterpret_cast<const uint2 *>(p);
      f[0] = __uint_as_float(r.x << 16);
      f[1] = __uint_as_float(r.x & 0xffff0000u);
      f[2] = __uint_as_float(r.y << 16);
      f[3] = __uint_as_float(r.y & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static void store(T *p, const float (&f)[V]) {
    if constexpr (V == 1) {
      *p = from_float<T>(f[0]);
    } else if constexpr (sizeof(T) * V == 16) {
      Elems<T, V> e;
      e.set(f);
      e.store(p);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
      *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
  }
};

__device__ __forceinline__ int conv_tokens(const ConvArgs &a, int b) {
  if (!a.lengths) return a.N;
  const long long n = a.len64 ? reinterpret_cast<const long long *>(a.lengths)[b]
                              : (long long)reinterpret_cast<const int *>(a.lengths)[b];
  return (int)(n < 0 ? 0 : n > a.N ? a.N : n);
}

template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int e, float (&w)[W][V], float (&bias)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.b ? a.b[e + v] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][v] = a.w[(size_t)(e + v) * W + k];
  }
}

// The input at position t >= -(W - 1) of a sequence: of the state before 0.
template <typename T, int V, int W>
__device__ __forceinline__ void input_at(const ConvArgs &a, int b, int e, int t, float (&f)[V]) {
  if (t >= 0) {
    Chans<T, V>::load(reinterpret_cast<const T *>(a.x) + b * a.sx[0] + t * a.sx[1] + e, f);
  } else if (a.state_in) {
    Chans<T, V>::load(reinterpret_cast<const T *>(a.state_in) + ((size_t)b * (W - 1) + (W - 1 + t)) * a.E + e, f);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.f;
  }
}

// run: tokens of a thread, at least W - 1 (then only the first run reads the
// state, which state_out may be).
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const ConvArgs a, int run, int runs) {
  constexpr int U = 4;  // tokens whose loads are in flight
  pdl_launch_dependents();
  pdl_wait();
  const int nv = a.E / V, b = blockIdx.y;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nv * runs) return;
  const int r = (int)(i / nv), e = (int)(i - (long long)r * nv) * V;
  const int n = conv_tokens(a, b), t0 = r * run, t1 = min(a.N, t0 + run), live = min(n, t1);
  float w[W][V], bias[V], win[W][V];  // win[k]: the input W - 1 - k tokens before
  load_taps<V, W>(a, e, w, bias);
  if (t0 < live)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) input_at<T, V, W>(a, b, e, t0 - (W - 1) + k, win[k + 1]);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + e;
  T *y = reinterpret_cast<T *>(a.out) + b * a.so[0] + e;
  for (int t = t0; t < live; t += U) {
    float in[U][V];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (t + j < live) Chans<T, V>::load(x + (t + j) * a.sx[1], in[j]);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (t + j >= live) break;
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
        win[W - 1][v] = in[j][v];
        float s = bias[v];
#pragma unroll
        for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[k][v], s);
        o[v] = a.silu ? silu(s) : s;
      }
      Chans<T, V>::store(y + (t + j) * a.so[1], o);
    }
  }
  const float zero[V] = {};
  for (int t = max(t0, live); t < t1; ++t) Chans<T, V>::store(y + t * a.so[1], zero);
  if (r == 0 && a.state_out) {
    float s[W - 1][V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) input_at<T, V, W>(a, b, e, n - (W - 1) + k, s[k]);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      Chans<T, V>::store(reinterpret_cast<T *>(a.state_out) + ((size_t)b * (W - 1) + k) * a.E + e, s[k]);
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
conv_bwd_kernel(const ConvArgs a, int run, int runs, float *__restrict__ part) {
  constexpr int U = 4;
  pdl_launch_dependents();
  pdl_wait();
  const int nv = a.E / V, b = blockIdx.y;
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (long long)nv * runs) return;
  const int r = (int)(i / nv), e = (int)(i - (long long)r * nv) * V;
  const int n = conv_tokens(a, b), t0 = r * run, t1 = min(a.N, t0 + run);
  float w[W][V], bias[V], win[W][V], d[W][V], dw[W][V], db[V];  // d[k]: of the token k before
  load_taps<V, W>(a, e, w, bias);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) win[k][v] = d[k][v] = dw[k][v] = 0.f;
  }
  if (t0 < n)
#pragma unroll
    for (int k = 0; k < W - 1; ++k) input_at<T, V, W>(a, b, e, t0 - (W - 1) + k, win[k + 1]);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + e;
  const T *dy = reinterpret_cast<const T *>(a.dy) + b * a.sg[0] + e;
  T *dx = reinterpret_cast<T *>(a.out) + b * a.so[0] + e;
  // Token t's d, and with it dx of token t - (W - 1), up to the run's last.
  for (int t = t0; t < t1 + W - 1; t += U) {
    float in[U][V], gr[U][V];
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (t + j < min(n, t1 + W - 1)) {
        Chans<T, V>::load(x + (t + j) * a.sx[1], in[j]);
        Chans<T, V>::load(dy + (t + j) * a.sg[1], gr[j]);
      }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int at = t + j, o = at - (W - 1);
      if (at >= t1 + W - 1) break;
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = W - 1; k > 0; --k) d[k][v] = d[k - 1][v];
        if (at < n) {
#pragma unroll
          for (int k = 0; k < W - 1; ++k) win[k][v] = win[k + 1][v];
          win[W - 1][v] = in[j][v];
          float dv = gr[j][v];
          if (a.silu) {
            float s = bias[v];
#pragma unroll
            for (int k = 0; k < W; ++k) s = fmaf(w[k][v], win[k][v], s);
            const float sg = sigmoid(s);
            dv *= sg * fmaf(s, 1.f - sg, 1.f);
          }
          d[0][v] = dv;
          if (at < t1) {
            db[v] += dv;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][v] = fmaf(dv, win[k][v], dw[k][v]);
          }
        } else {
          d[0][v] = 0.f;
        }
        out[v] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) out[v] = fmaf(w[k][v], d[k][v], out[v]);
      }
      if (o >= t0 || (r == 0 && o < 0)) {
        // what the state after the sequence passes back to the last W - 1 inputs
        const int m = o - (n - (W - 1));
        if (a.dstate_out && m >= 0 && m < W - 1) {
          float s[V];
          Chans<T, V>::load(reinterpret_cast<const T *>(a.dstate_out) + ((size_t)b * (W - 1) + m) * a.E + e, s);
#pragma unroll
          for (int v = 0; v < V; ++v) out[v] += s[v];
        }
        if (o >= 0)
          Chans<T, V>::store(dx + o * a.so[1], out);
        else if (a.dstate_in)
          Chans<T, V>::store(reinterpret_cast<T *>(a.dstate_in) + ((size_t)b * (W - 1) + W - 1 + o) * a.E + e, out);
      }
    }
  }
  if (!part) return;
  const size_t row = (size_t)b * runs + r, rows = (size_t)a.B * runs;
  float *pb = part + rows * a.E * W;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    pb[row * a.E + e + v] = db[v];
#pragma unroll
    for (int k = 0; k < W; ++k) part[(row * a.E + e + v) * W + k] = dw[k][v];
  }
}

bool aligned(const void *p, const long long s[2], int B, int N, int bytes, int esz) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (N <= 1 || s[1] * esz % bytes == 0) &&
         (B <= 1 || s[0] * esz % bytes == 0);
}

// 32 tokens a thread (the W - 1 at its ends are read twice), fewer where that
// leaves less than 1024 threads an SM.
int run_of(const ConvArgs &a, int nv, int most) {
  int run = most;
  while (run > 4 && (long long)nv * a.B * ((a.N + run - 1) / run) < 1024LL * device_sms()) run /= 2;
  return run;
}
int runs_of(int N, int run) { return std::max(1, (N + run - 1) / run); }

template <typename T, int V, int W>
cudaError_t fwd(const ConvArgs &a, cudaStream_t st) {
  const int nv = a.E / V, run = run_of(a, nv, 32), runs = runs_of(a.N, run);
  const dim3 grid((unsigned)(((long long)nv * runs + kThreads - 1) / kThreads), a.B);
  return launch_k(conv_fwd_kernel<T, V, W>, grid, dim3(kThreads), 0, st, true, a, run, runs);
}

template <typename T, int V, int W>
cudaError_t bwd(const ConvArgs &a, float *part, cudaStream_t st) {
  const int runs = conv_bwd_runs(a) / a.B, run = std::max(4, (a.N + runs - 1) / runs);
  const dim3 grid((unsigned)(((long long)(a.E / V) * runs + kThreads - 1) / kThreads), a.B);
  return launch_k(conv_bwd_kernel<T, V, W>, grid, dim3(kThreads), 0, st, true, a, run, runs, part);
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

cudaError_t launch_conv_fwd(const ConvArgs &a, int bf16, cudaStream_t st) {
  const int esz = bf16 ? 2 : 4;
  const bool v = a.E * esz % 16 == 0 && aligned(a.x, a.sx, a.B, a.N, 16, esz) && aligned(a.out, a.so, a.B, a.N, 16, esz) &&
                 reinterpret_cast<uintptr_t>(a.state_in) % 16 == 0 && reinterpret_cast<uintptr_t>(a.state_out) % 16 == 0;
  if (bf16) return v ? fwd_taps<__nv_bfloat16, 8>(a, st) : fwd_taps<__nv_bfloat16, 1>(a, st);
  return v ? fwd_taps<float, 4>(a, st) : fwd_taps<float, 1>(a, st);
}

// Runs of tokens over all sequences (at most 64 tokens each, fewer where that
// leaves less than 1024 threads an SM).
int conv_bwd_runs(const ConvArgs &a) {
  const int nv = std::max(1, a.E / 4);
  return runs_of(a.N, run_of(a, nv, 64)) * a.B;
}

cudaError_t launch_conv_bwd(const ConvArgs &a, int bf16, float *part, cudaStream_t st) {
  const int esz = bf16 ? 2 : 4, by = 4 * esz;
  const bool v = a.E % 4 == 0 && aligned(a.x, a.sx, a.B, a.N, by, esz) && aligned(a.dy, a.sg, a.B, a.N, by, esz) &&
                 aligned(a.out, a.so, a.B, a.N, by, esz) && reinterpret_cast<uintptr_t>(a.state_in) % by == 0 &&
                 reinterpret_cast<uintptr_t>(a.dstate_in) % by == 0 && reinterpret_cast<uintptr_t>(a.dstate_out) % by == 0;
  if (bf16) return v ? bwd_taps<__nv_bfloat16, 4>(a, part, st) : bwd_taps<__nv_bfloat16, 1>(a, part, st);
  return v ? bwd_taps<float, 4>(a, part, st) : bwd_taps<float, 1>(a, part, st);
}

}  // namespace ret
