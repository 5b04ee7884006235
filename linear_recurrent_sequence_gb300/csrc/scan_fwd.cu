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

template <int L>
struct FwdSmem {
  float4 du[2][Block<L>::kTile][Block<L>::kChannels];  // delta, delta, u, u
  float bm[2][Block<L>::kTile][Block<L>::SP], cm[2][Block<L>::kTile][Block<L>::SP];
  float ysum[2][Block<L>::kTile][Block<L>::kChannels];
};

// Half of the CTA's warps walk the recurrence; the others load the tokens two
// tiles ahead, work out step sizes and inputs, and finish the outputs of the
// tile before: with one sequence an SM has no more than one recurrence warp a
// scheduler, and everything else that a token needs runs beside it.
// kStates: only the states that the segments leave behind.
template <typename T, int L, bool kStates, bool kPair>
__global__ void __launch_bounds__(kThreads, 2)
scan_fwd_kernel(const ScanArgs a, const ScanSegs seg) {
  using K = Block<L>;
  constexpr int CC = K::kChannels, TT = K::kTile, SP = K::SP;
  extern __shared__ __align__(16) uint8_t dyn[];
  FwdSmem<L> &sm = *reinterpret_cast<FwdSmem<L> *>(dyn);
  pdl_wait();
  const int per = K::per_group(a.E, a.G), Eg = a.E / a.G;
  const int group = blockIdx.x / per, c0 = (blockIdx.x - group * per) * CC;  // within the group
  const int b = blockIdx.z, k = blockIdx.y;
  const int n = tokens_of(a, b), t0 = k * seg.len, t1 = min(a.N, t0 + seg.len), live = min(t1, n);
  const int tiles = live > t0 ? (live - t0 + TT - 1) / TT : 0;

  if (threadIdx.x < kScan) {
    // ---- four states of a channel
    const int tid = threadIdx.x, ci = tid / L, s0 = tid % L * 4;
    const bool own = c0 + ci < Eg, vec = a.S % 4 == 0;
    const int e = group * Eg + min(c0 + ci, Eg - 1);
    const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
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
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const int buf = i & 1;
      // (16 tokens' outputs are stored at once: a store between them would hold
      // back the loads behind it, and a warp alone on its scheduler has nothing
      // else to do; 76 cycles a token with stores every 4 tokens)
      constexpr int GT = TT < 16 ? TT : 16;
#pragma unroll
      for (int q = 0; q < TT; q += GT) {
        float yq[GT / 4][4];
#pragma unroll
        for (int j = 0; j < GT; ++j) {
          const float4 v = sm.du[buf][q + j][ci];
          const float4 B4 = *reinterpret_cast<const float4 *>(&sm.bm[buf][q + j][s0]);
          const float2 dd = make_float2(v.x, v.y), uu = make_float2(v.z, v.w);
          const float2 w01 = tc::mul2(dd, A01), w23 = tc::mul2(dd, A23);
          const float2 i01 = tc::mul2(uu, make_float2(B4.x, B4.y)), i23 = tc::mul2(uu, make_float2(B4.z, B4.w));
          h01 = tc::fma2(make_float2(ex2(w01.x), ex2(w01.y)), h01, i01);
          h23 = tc::fma2(make_float2(ex2(w23.x), ex2(w23.y)), h23, i23);
          if (!kStates) {
            const float4 C4 = *reinterpret_cast<const float4 *>(&sm.cm[buf][q + j][s0]);
            const float2 s = tc::fma2(h23, make_float2(C4.z, C4.w), tc::mul2(h01, make_float2(C4.x, C4.y)));
            yq[j / 4][j % 4] = s.x + s.y;
            if (j % 4 == 3) share_sums<4, L>(yq[j / 4]);
          }
        }
        if (!kStates) {
          constexpr int M = L < 4 ? L : 4;
          if (tid % L < M)
#pragma unroll
            for (int i4 = 0; i4 < GT / 4; ++i4)
#pragma unroll
              for (int j = 0; j < 4 / M; ++j) sm.ysum[buf][q + i4 * 4 + tid % M * (4 / M) + j][ci] = yq[i4][j];
        }
      }
      __syncthreads();
    }
    pdl_launch_dependents();
    const float4 h4 = make_float4(h01.x, h01.y, h23.x, h23.y);
    if (kStates) {
      if (own) store_states(seg.loc + (size_t)k * a.B * a.E * a.S + row, s0, a.S, vec, h4);
    } else if (k == seg.count - 1 && own && a.h_out) {
      store_states(a.h_out + row, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0, h4);
    }
    if (kStates) __syncthreads();
    return;
  }

  // ---- two channels' tokens, NP of each tile
  constexpr int NP = TT * CC / 2 / kLoad, TS = 2 * kLoad / CC;  // pairs a thread; tokens between them
  constexpr int NB = (TT * SP + kLoad - 1) / kLoad;
  static_assert(NP * kLoad * 2 == TT * CC && NP * TS == TT, "whole tiles");
  const int tid = threadIdx.x - kScan, lc = tid % (CC / 2) * 2, lt = tid / (CC / 2);
  const int there = min(2, max(0, Eg - c0 - lc));  // channels of this pair
  const int le = group * Eg + min(c0 + lc, Eg - 1);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + le;
  const T *dt = reinterpret_cast<const T *>(a.dt) + b * a.sdt[0] + le;
  const T *z = kStates || !a.z ? nullptr : reinterpret_cast<const T *>(a.z) + b * a.sz[0] + le;
  const T *Bp = reinterpret_cast<const T *>(a.Bm) + b * a.sB[0] + group * a.sB[2];
  const T *Cp = reinterpret_cast<const T *>(a.Cm) + b * a.sC[0] + group * a.sC[2];
  T *y = reinterpret_cast<T *>(a.y) + b * a.sy[0] + le;
  const int l1 = there > 1;
  const float bias[2] = {a.bias ? a.bias[le] : 0.f, a.bias ? a.bias[le + l1] : 0.f};
  const float Dv[2] = {!kStates && a.D ? a.D[le] : 0.f, !kStates && a.D ? a.D[le + l1] : 0.f};
  float dsum[2] = {0.f, 0.f};

  struct Raw {
    Two<T> x[NP], z[NP], d[NP];
    T B[NB], C[NB];
  };
  struct Kept {
    Two<T> x[NP], z[NP];
  };
  auto load = [&](int i, Raw &r) {
    if (i >= tiles) return;
    const int t = t0 + i * TT;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int at = t + lt + j * TS, m = at < live ? there : 0;
      r.x[j] = load_two<T, kPair>(x + at * a.sx[1], m);
      r.d[j] = load_two<T, kPair>(dt + at * a.sdt[1], m);
      if (!kStates) r.z[j] = load_two<T, kPair>(z + at * a.sz[1], z ? m : 0);
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int o = tid + j * kLoad, at = t + o / SP, s = o % SP;
      const bool in = (NB * kLoad == TT * SP || o < TT * SP) && at < live && s < a.S;
      r.B[j] = in ? Bp[at * a.sB[1] + s] : from_float<T>(0.f);
      if (!kStates) r.C[j] = in ? Cp[at * a.sC[1] + s] : from_float<T>(0.f);
    }
  };
  // What was loaded for tile i becomes delta, u, B and C; past the end delta and
  // u are 0 and leave the state as it is.
  auto put = [&](int i, const Raw &r) {
    const int buf = i & 1, t = t0 + i * TT;
    float part[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int at = lt + j * TS;
      const float xs[2] = {to_float(r.x[j].a), to_float(r.x[j].b)};
      float d[2] = {to_float(r.d[j].a) + bias[0], to_float(r.d[j].b) + bias[1]};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (a.softplus) d[c] = softplus(d[c]);
        if (!(c < there && t + at < live)) d[c] = 0.f;
        const float u = d[c] * xs[c];
        sm.du[buf][at][lc + c] = make_float4(d[c], d[c], u, u);
        if (kStates) part[c] += d[c];
      }
    }
    if (kStates) {
      dsum[0] += part[0];
      dsum[1] += part[1];
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int o = tid + j * kLoad;
      if (NB * kLoad == TT * SP || o < TT * SP) {
        (&sm.bm[buf][0][0])[o] = to_float(r.B[j]);
        if (!kStates) (&sm.cm[buf][0][0])[o] = to_float(r.C[j]);
      }
    }
  };
  auto finish = [&](int i, const Kept &r) {
    const int buf = i & 1, t = t0 + i * TT;
#pragma unroll
    for (int j = 0; j < (kStates ? 0 : NP); ++j) {
      const int at = lt + j * TS;
      const float2 s = *reinterpret_cast<const float2 *>(&sm.ysum[buf][at][lc]);
      float v0 = fmaf(Dv[0], to_float(r.x[j].a), s.x), v1 = fmaf(Dv[1], to_float(r.x[j].b), s.y);
      if (z) {
        v0 *= silu(to_float(r.z[j].a));
        v1 *= silu(to_float(r.z[j].b));
      }
      const bool in = t + at < live;
      if (t + at < t1) store_two<T, kPair>(y + (t + at) * a.sy[1], there, in ? v0 : 0.f, in ? v1 : 0.f);
    }
  };
  auto keep = [&](const Raw &r, Kept &q) {
#pragma unroll
    for (int j = 0; j < (kStates ? 0 : NP); ++j) {
      q.x[j] = r.x[j];
      q.z[j] = r.z[j];
    }
  };

  // Two buffers of what is on its way, each known by name (a copy from one to the
  // other would wait for the loads).
  Raw even, odd;
  Kept cur, done;
  load(0, even);
  load(1, odd);
  if (tiles > 0) put(0, even);
  keep(even, cur);
  __syncthreads();
  auto turn = [&](int i, Raw &next, Raw &free) {  // next: tile i + 1
    load(i + 2, free);
    if (i > 0) finish(i - 1, done);
    if (i + 1 < tiles) put(i + 1, next);
    __syncthreads();
    done = cur;
    keep(next, cur);
  };
  for (int i = 0; i < tiles; i += 2) {
    turn(i, odd, even);
    if (i + 1 < tiles) turn(i + 1, even, odd);
  }
  if (tiles > 0) finish(tiles - 1, done);
  pdl_launch_dependents();
  if (!kStates) {  // whole tiles past the sequence's end
    for (int at = t0 + tiles * TT + lt; at < t1; at += TS) store_two<T, kPair>(y + at * a.sy[1], there, 0.f, 0.f);
  } else {
    // the loaders' sums of a channel, in order (the walk over the tiles is over)
    float *red = &sm.ysum[0][0][0];
    red[lt * CC + lc] = dsum[0];
    red[lt * CC + lc + 1] = dsum[1];
    __syncthreads();
    if (tid < CC && c0 + tid < Eg) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < TS; ++i) s += red[i * CC + tid];
      seg.sum[((size_t)k * a.B + b) * a.E + group * Eg + c0 + tid] = s;
    }
  }
}

// One token.  A lane has four states of R sequences' same channel, so that A is
// read once for them; what a sequence's channel needs once (step size, gate,
// output) is shared out over the channel's lanes.
constexpr int kStepThreads = 256;

template <typename T, int L, int R, bool kVec>
__global__ void __launch_bounds__(kStepThreads)
scan_step_kernel(const ScanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int CC = kStepThreads / L, M = L < R ? L : R, NR = R / M;  // lanes that have sequences, of each NR
  const int lane = threadIdx.x & 31, ci = threadIdx.x / L, sub = threadIdx.x % L, s0 = sub * 4;
  const int c = blockIdx.x * CC + ci, e = min(c, a.E - 1), g = e / (a.E / a.G);
  const bool own = c < a.E, vec = a.S % 4 == 0;
  const bool va = vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0;
  const bool vi = vec && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0;
  const bool vo = vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0;
  const int b0 = blockIdx.y * R, there = min(R, a.B - b0);
  const size_t row = ((size_t)b0 * a.E + e) * a.S, step = (size_t)a.E * a.S;
  float4 h[R];
  Four<T> Br[R], Cr[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < there) h[r] = load_states(a.h_in + row + r * step, s0, a.S, vi);
  {
    const T *Bp = reinterpret_cast<const T *>(a.Bm) + b0 * a.sB[0] + g * a.sB[2] + s0;
    const T *Cp = reinterpret_cast<const T *>(a.Cm) + b0 * a.sC[0] + g * a.sC[2] + s0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < there) {
        Br[r] = load_four<T, kVec>(Bp + r * a.sB[0], a.S - s0);
        Cr[r] = load_four<T, kVec>(Cp + r * a.sC[0], a.S - s0);
      }
  }
  // this lane's sequences: sub NR .. sub NR + NR - 1
  const float bias = a.bias ? a.bias[e] : 0.f, Dv = a.D ? a.D[e] : 0.f;
  float x[NR], d[NR], gate[NR];
#pragma unroll
  for (int m = 0; m < NR; ++m) {
    const int b = b0 + min(sub % M * NR + m, there - 1);
    x[m] = to_float(reinterpret_cast<const T *>(a.x)[b * a.sx[0] + e]);
    d[m] = to_float(reinterpret_cast<const T *>(a.dt)[b * a.sdt[0] + e]) + bias;
    gate[m] = a.z ? to_float(reinterpret_cast<const T *>(a.z)[b * a.sz[0] + e]) : 0.f;
  }
  const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, va);
  const float As[4] = {A4.x * kLog2e, A4.y * kLog2e, A4.z * kLog2e, A4.w * kLog2e};
#pragma unroll
  for (int m = 0; m < NR; ++m) {
    if (a.softplus) d[m] = softplus(d[m]);
    gate[m] = a.z ? silu(gate[m]) : 1.f;
  }
  float sum[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int from = lane / L * L + r / NR;
    const float dr = __shfl_sync(0xffffffffu, d[r % NR], from);
    const float u = dr * __shfl_sync(0xffffffffu, x[r % NR], from);
    float hs[4] = {h[r].x, h[r].y, h[r].z, h[r].w};
    sum[r] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hs[j] = fmaf(ex2(dr * As[j]), hs[j], u * to_float(Br[r].v[j]));
      sum[r] = fmaf(hs[j], to_float(Cr[r].v[j]), sum[r]);
    }
    if (own && r < there) store_states(a.h_out + row + r * step, s0, a.S, vo, make_float4(hs[0], hs[1], hs[2], hs[3]));
  }
  share_sums<R, L>(sum);
#pragma unroll
  for (int m = 0; m < NR; ++m) {
    const int r = sub * NR + m;
    if (own && r < there)
      reinterpret_cast<T *>(a.y)[(b0 + r) * a.sy[0] + e] = from_float<T>(fmaf(Dv, x[m], sum[m]) * gate[m]);
  }
}

// Pairs of channels are read and written at once where every row of every
// tensor (and every block of channels) begins on a pair's boundary.
bool pairs_ok(const ScanArgs &a, int esz, bool states) {
  return a.E / a.G % 2 == 0 && rows_on(a, a.x, a.sx, 2, esz) && rows_on(a, a.dt, a.sdt, 2, esz) &&
         (states || (rows_on(a, a.z, a.sz, 2, esz) && rows_on(a, a.y, a.sy, 2, esz)));
}

template <typename T, int L, bool kStates, bool kPair>
cudaError_t scan_with(const ScanArgs &a, const ScanSegs &seg, int segs, cudaStream_t st) {
  static std::atomic<unsigned> done{0};
  auto kern = scan_fwd_kernel<T, L, kStates, kPair>;
  const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.G * Block<L>::per_group(a.E, a.G), segs, a.B);
  return launch_k(kern, grid, dim3(kThreads), sizeof(FwdSmem<L>), st, true, a, seg);
}

template <typename T, bool kStates>
cudaError_t scan_any(const ScanArgs &a, const ScanSegs &seg, int segs, cudaStream_t st) {
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    return pairs_ok(a, sizeof(T), kStates) ? scan_with<T, L, kStates, true>(a, seg, segs, st)
                                           : scan_with<T, L, kStates, false>(a, seg, segs, st);
  });
}

template <typename T, int R>
cudaError_t step_any(const ScanArgs &a, cudaStream_t st) {
  auto on = [&](const void *p, const long long s[3]) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && (a.B == 1 || s[0] % 4 == 0) && (a.G == 1 || s[2] % 4 == 0);
  };
  const bool vec = a.S % 4 == 0 && on(a.Bm, a.sB) && on(a.Cm, a.sC);
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value, CC = kStepThreads / L;
    const dim3 grid((a.E + CC - 1) / CC, (a.B + R - 1) / R);
    return vec ? launch_k(scan_step_kernel<T, L, R, true>, grid, dim3(kStepThreads), 0, st, true, a)
               : launch_k(scan_step_kernel<T, L, R, false>, grid, dim3(kStepThreads), 0, st, true, a);
  });
}

}  // namespace

// Segments only where a sequence's channels leave most SMs without a CTA: the
// exponentials of all but the last segment are then taken twice.
ScanSegs scan_fwd_plan(const ScanArgs &a) {
  ScanSegs s;
  s.len = std::max(a.N, 1);
  int tile = 1;
  long long ctas = 1;
  by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    tile = Block<L>::kTile;
    ctas = (long long)a.G * Block<L>::per_group(a.E, a.G) * a.B;
    return cudaSuccess;
  });
  const int sms = device_sms();
  if (ctas * 2 > sms || a.N < 8 * tile) return s;
  const long long want = std::min<long long>(2 * sms / std::max(ctas, 1LL), a.N / (4 * tile));
  s.len = (int)((a.N + want - 1) / want + tile - 1) / tile * tile;
  s.count = (a.N + s.len - 1) / s.len;
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
  // Four sequences a thread once one each would give every SM over 16 CTAs.
  const long long ctas = ((long long)a.E * lanes_of(a.S) + kStepThreads - 1) / kStepThreads * a.B;
  if (ctas >= 16LL * device_sms()) return bf16 ? step_any<__nv_bfloat16, 4>(a, st) : step_any<float, 4>(a, st);
  return bf16 ? step_any<__nv_bfloat16, 1>(a, st) : step_any<float, 1>(a, st);
}

}  // namespace ret
