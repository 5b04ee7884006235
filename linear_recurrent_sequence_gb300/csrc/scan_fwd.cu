// The selective scan, forward (a state space model whose step size, input and
// output vectors depend on the token):
//   delta = softplus(dt + bias),  h_t[s] = e^(delta_t A[s]) h_{t-1}[s] + delta_t x_t B_t[s],
//   y_t = (sum_s C_t[s] h_t[s] + D x_t) silu(z_t)
// for each channel on its own; A is the channel's, B and C those of its group.
// fp32 arithmetic and states for bf16 and fp32 tensors.
//
// A channel's states are shared out over L neighbouring lanes, four a lane, in
// registers for the whole sequence.  Per token and state: one exponential and
// four operations, three of them on packed pairs.  The step sizes delta and
// u = delta x are worked out once per token and channel by the thread that
// loads them, and handed on in shared memory together with B and C.
#include <algorithm>

#include "scan.cuh"

namespace ret {

namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kTile = 16;  // tokens at a time

// Channels of a CTA; grid.x counts the blocks of all groups.
template <int L>
struct Block {
  static constexpr int kChannels = kThreads / L;
  static __host__ __device__ int per_group(int E, int G) { return (E / G + kChannels - 1) / kChannels; }
};

// kStates: only the states that the segments leave behind.
template <typename T, int L, bool kStates>
__global__ void __launch_bounds__(kThreads)
scan_fwd_kernel(const ScanArgs a, const ScanSegs seg) {
  constexpr int CC = Block<L>::kChannels, NE = kTile / L, SP = 4 * L, NB = (kTile * SP + kThreads - 1) / kThreads;
  __shared__ __align__(16) float2 du[2][kTile][CC];
  __shared__ __align__(16) float bm[2][kTile][SP], cm[kStates ? 1 : 2][kTile][SP];
  __shared__ float ysum[kStates ? 1 : 2][kTile][CC];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, per = Block<L>::per_group(a.E, a.G), Eg = a.E / a.G;
  const int group = blockIdx.x / per, c0 = (blockIdx.x - group * per) * CC;  // within the group
  const int b = blockIdx.z, k = blockIdx.y;
  const int n = tokens_of(a, b), t0 = k * seg.len, t1 = min(a.N, t0 + seg.len), live = min(t1, n);

  // As owner of four states of a channel ...
  const int ci = tid / L, s0 = tid % L * 4;
  const bool own = c0 + ci < Eg;
  const int e = group * Eg + min(c0 + ci, Eg - 1);
  const bool vec = a.S % 4 == 0;
  float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
  const float2 A01 = make_float2(A4.x * kLog2e, A4.y * kLog2e), A23 = make_float2(A4.z * kLog2e, A4.w * kLog2e);
  float2 h01 = both(0.f), h23 = both(0.f);
  const size_t row = ((size_t)b * a.E + e) * a.S;
  if (!kStates) {
    // the state that the segments before this one leave behind
    if (a.h_in) {
      const float4 h = load_states(a.h_in + row, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0);
      h01 = make_float2(h.x, h.y);
      h23 = make_float2(h.z, h.w);
    }
    for (int i = 0; i < k; ++i) {
      const float2 d = both(seg.sum[((size_t)i * a.B + b) * a.E + e]);
      const float4 l = load_states(seg.loc + (size_t)i * a.B * a.E * a.S + row, s0, a.S, vec);
      const float2 w01 = tc::mul2(d, A01), w23 = tc::mul2(d, A23);
      h01 = tc::fma2(make_float2(ex2(w01.x), ex2(w01.y)), h01, make_float2(l.x, l.y));
      h23 = tc::fma2(make_float2(ex2(w23.x), ex2(w23.y)), h23, make_float2(l.z, l.w));
    }
  }

  // ... and as loader of one channel's tokens, NE of each tile.
  const int lc = tid % CC, lt = tid / CC;
  const bool there = c0 + lc < Eg;
  const int le = group * Eg + min(c0 + lc, Eg - 1);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + le;
  const T *dt = reinterpret_cast<const T *>(a.dt) + b * a.sdt[0] + le;
  const T *z = kStates || !a.z ? nullptr : reinterpret_cast<const T *>(a.z) + b * a.sz[0] + le;
  const T *Bp = reinterpret_cast<const T *>(a.Bm) + b * a.sB[0] + group * a.sB[2];
  const T *Cp = reinterpret_cast<const T *>(a.Cm) + b * a.sC[0] + group * a.sC[2];
  T *y = reinterpret_cast<T *>(a.y) + b * a.sy[0] + le;
  const float bias = a.bias ? a.bias[le] : 0.f, Dv = !kStates && a.D ? a.D[le] : 0.f;
  T xn[NE], dn[NE], zn[NE], bn[NB], cn[NB];
  float xc[NE], zc[NE];
  float dsum = 0.f;

  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int at = t + lt + i * L;
      const bool in = there && at < live;
      xn[i] = in ? x[at * a.sx[1]] : from_float<T>(0.f);
      dn[i] = in ? dt[at * a.sdt[1]] : from_float<T>(0.f);
      if (!kStates) zn[i] = z && in ? z[at * a.sz[1]] : from_float<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int j = tid + i * kThreads, at = t + j / SP, s = j % SP;
      const bool in = (NB * kThreads == kTile * SP || j < kTile * SP) && at < live && s < a.S;
      bn[i] = in ? Bp[at * a.sB[1] + s] : from_float<T>(0.f);
      if (!kStates) cn[i] = in ? Cp[at * a.sC[1] + s] : from_float<T>(0.f);
    }
  };
  // What was loaded for the tile at t becomes delta, u, B and C; past the end
  // delta and u are 0 and leave the state as it is.
  auto put = [&](int t, int buf) {
    float part = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int at = lt + i * L;
      float d = to_float(dn[i]) + bias;
      if (a.softplus) d = softplus(d);
      if (!(there && t + at < live)) d = 0.f;
      const float xf = to_float(xn[i]);
      du[buf][at][lc] = make_float2(d, d * xf);
      if (kStates) part += d;
      if (!kStates) {
        xc[i] = xf;
        zc[i] = to_float(zn[i]);
      }
    }
    dsum += part;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int j = tid + i * kThreads;
      if (NB * kThreads == kTile * SP || j < kTile * SP) {
        (&bm[buf][0][0])[j] = to_float(bn[i]);
        if (!kStates) (&cm[buf][0][0])[j] = to_float(cn[i]);
      }
    }
  };

  float xo[NE], zo[NE];
  int buf = 0;
  load(t0);
  put(t0, 0);
  __syncthreads();
  for (int t = t0; t < live; t += kTile, buf ^= 1) {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      xo[i] = xc[i];
      zo[i] = zc[i];
    }
    const bool more = t + kTile < live;
    if (more) load(t + kTile);
#pragma unroll
    for (int q = 0; q < kTile; q += 4) {
      float yq[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = du[buf][q + j][ci];
        const float4 B4 = *reinterpret_cast<const float4 *>(&bm[buf][q + j][s0]);
        const float2 dd = both(v.x), uu = both(v.y);
        const float2 w01 = tc::mul2(dd, A01), w23 = tc::mul2(dd, A23);
        const float2 i01 = tc::mul2(uu, make_float2(B4.x, B4.y)), i23 = tc::mul2(uu, make_float2(B4.z, B4.w));
        h01 = tc::fma2(make_float2(ex2(w01.x), ex2(w01.y)), h01, i01);
        h23 = tc::fma2(make_float2(ex2(w23.x), ex2(w23.y)), h23, i23);
        if (!kStates) {
          const float4 C4 = *reinterpret_cast<const float4 *>(&cm[buf][q + j][s0]);
          const float2 s = tc::fma2(h23, make_float2(C4.z, C4.w), tc::mul2(h01, make_float2(C4.x, C4.y)));
          yq[j] = s.x + s.y;
        }
      }
      if (!kStates) {
        share_sums<4, L>(yq);
        constexpr int M = L < 4 ? L : 4;
#pragma unroll
        for (int j = 0; j < 4 / M; ++j)
          if (tid % L < M) ysum[buf][q + tid % M * (4 / M) + j][ci] = yq[j];
      }
    }
    if (more) put(t + kTile, buf ^ 1);
    __syncthreads();
    if (!kStates) {
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        const int at = t + lt + i * L;
        if (there && at < t1) {
          float v = fmaf(Dv, xo[i], ysum[buf][lt + i * L][lc]);
          if (z) v *= silu(zo[i]);
          y[at * a.sy[1]] = from_float<T>(at < live ? v : 0.f);
        }
      }
    }
  }
  if (!kStates) {  // whole tiles past the sequence's end
    const int done = live > t0 ? t0 + (live - t0 + kTile - 1) / kTile * kTile : t0;
    for (int at = done + lt; at < t1; at += L)
      if (there) y[at * a.sy[1]] = from_float<T>(0.f);
  }
  if (kStates) {
    if (own) store_states(seg.loc + (size_t)k * a.B * a.E * a.S + row, s0, a.S, vec, make_float4(h01.x, h01.y, h23.x, h23.y));
    // the loaders' sums of a channel, in order
    __syncthreads();
    float *red = reinterpret_cast<float *>(&du[0][0][0]);
    red[lt * CC + lc] = dsum;
    __syncthreads();
    if (tid < CC && there) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < L; ++i) s += red[i * CC + tid];
      seg.sum[((size_t)k * a.B + b) * a.E + le] = s;
    }
  } else if (k == seg.count - 1 && own && a.h_out) {
    store_states(a.h_out + row, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0,
                 make_float4(h01.x, h01.y, h23.x, h23.y));
  }
}

// One token.  A lane has four states of R sequences' same channel, so that A
// is read once for them.
constexpr int kStepThreads = 256;

template <typename T, int L, int R>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(const ScanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int CC = kStepThreads / L;
  const int ci = threadIdx.x / L, s0 = threadIdx.x % L * 4;
  const int c = blockIdx.x * CC + ci, e = min(c, a.E - 1), g = e / (a.E / a.G);
  const bool own = c < a.E, vec = a.S % 4 == 0;
  const bool va = vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0;
  const bool vi = vec && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0;
  const bool vo = vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0;
  const int b0 = blockIdx.y * R;
  float4 h[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = min(b0 + r, a.B - 1);
    h[r] = load_states(a.h_in + ((size_t)b * a.E + e) * a.S, s0, a.S, vi);
  }
  const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, va);
  const float bias = a.bias ? a.bias[e] : 0.f, Dv = a.D ? a.D[e] : 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int b = min(b0 + r, a.B - 1);
    const float x = to_float(reinterpret_cast<const T *>(a.x)[b * a.sx[0] + e]);
    float d = to_float(reinterpret_cast<const T *>(a.dt)[b * a.sdt[0] + e]) + bias;
    if (a.softplus) d = softplus(d);
    const T *Bp = reinterpret_cast<const T *>(a.Bm) + b * a.sB[0] + g * a.sB[2];
    const T *Cp = reinterpret_cast<const T *>(a.Cm) + b * a.sC[0] + g * a.sC[2];
    const float u = d * x, w = d * kLog2e;
    float hs[4] = {h[r].x, h[r].y, h[r].z, h[r].w};
    const float As[4] = {A4.x, A4.y, A4.z, A4.w};
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = s0 + j < a.S;
      const float Bv = in ? to_float(Bp[s0 + j]) : 0.f, Cv = in ? to_float(Cp[s0 + j]) : 0.f;
      hs[j] = fmaf(ex2(w * As[j]), hs[j], u * Bv);
      s[0] = fmaf(hs[j], Cv, s[0]);
    }
    share_sums<1, L>(s);
    const bool mine = own && b0 + r < a.B;
    if (mine) store_states(a.h_out + ((size_t)b * a.E + e) * a.S, s0, a.S, vo, make_float4(hs[0], hs[1], hs[2], hs[3]));
    if (mine && s0 == 0) {
      float v = fmaf(Dv, x, s[0]);
      if (a.z) v *= silu(to_float(reinterpret_cast<const T *>(a.z)[b * a.sz[0] + e]));
      reinterpret_cast<T *>(a.y)[b * a.sy[0] + e] = from_float<T>(v);
    }
  }
}

// Lanes a channel: four states a lane.
int lanes_of(int S) {
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

template <typename T, bool kStates>
cudaError_t scan_any(const ScanArgs &a, const ScanSegs &seg, int segs, cudaStream_t st) {
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    const dim3 grid(a.G * Block<L>::per_group(a.E, a.G), segs, a.B);
    return launch_k(scan_fwd_kernel<T, L, kStates>, grid, dim3(kThreads), 0, st, true, a, seg);
  });
}

template <typename T>
cudaError_t step_any(const ScanArgs &a, cudaStream_t st) {
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value, CC = kStepThreads / L;
    const int nx = (a.E + CC - 1) / CC;
    if ((long long)nx * a.B >= 16LL * device_sms())
      return launch_k(scan_step_kernel<T, L, 4>, dim3(nx, (a.B + 3) / 4), dim3(kStepThreads), 0, st, true, a);
    return launch_k(scan_step_kernel<T, L, 1>, dim3(nx, a.B), dim3(kStepThreads), 0, st, true, a);
  });
}

}  // namespace

ScanSegs scan_fwd_plan(const ScanArgs &a) {
  ScanSegs s;
  s.len = std::max(a.N, 1);
  return s;
}

size_t scan_fwd_bytes(const ScanArgs &a) {
  return (size_t)(scan_fwd_plan(a).count - 1) * a.B * a.E * (a.S + 1) * sizeof(float);
}

cudaError_t launch_scan_states(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st) {
  return bf16 ? scan_any<__nv_bfloat16, true>(a, seg, seg.count - 1, st)
              : scan_any<float, true>(a, seg, seg.count - 1, st);
}

cudaError_t launch_scan_fwd(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st) {
  return bf16 ? scan_any<__nv_bfloat16, false>(a, seg, seg.count, st)
              : scan_any<float, false>(a, seg, seg.count, st);
}

cudaError_t launch_scan_step(const ScanArgs &a, int bf16, cudaStream_t st) {
  return bf16 ? step_any<__nv_bfloat16>(a, st) : step_any<float>(a, st);
}

}  // namespace ret
