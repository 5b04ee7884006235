// Gradients of the selective scan.  With ds = dy silu(z) (dy without z) and
// p_t = e^(delta_t A) h_{t-1}, so that h_t = p_t + u_t B_t, u = delta x:
//   g_t = C_t ds_t + e^(delta_{t+1} A) g_{t+1}      (dL/dh_t, per channel and state)
//   dC_t = sum_channels ds_t h_t,   dB_t = sum_channels u_t g_t,
//   q_t = sum_s g_t B_t,  r_t = sum_s g_t p_t A,   dA = sum_t g_t p_t delta_t,
//   dx_t = delta_t q_t + D ds_t,  ddelta_t = x_t q_t + r_t,  ddt = ddelta softplus'(dt + bias),
//   dz_t = dy_t (sum_s C_t h_t + D x_t) silu'(z_t),  dD = sum ds x,  dbias = sum ddt.
// fp32 arithmetic.
//
// The sequence is cut into chunks.  One pass over each chunk alone gives what
// it adds to the state after it and to the gradient before it (both walk the
// same exponentials, forwards: the second is sum_t (e^(A (delta_1 + .. + delta_t)))
// C_t ds_t).  A short pass over the chunks joins them, and then every chunk has
// its own CTA: forwards once, keeping the state at every 8th token, then tile
// by tile backwards with 8 tokens' decays and states in registers (running a
// state backwards instead would divide by decays that underflow).
// A thread has four states of two neighbouring channels; sums over a channel's
// states are shared out over its L lanes, sums over channels over the others.
#include <algorithm>

#include "scan.cuh"

namespace ret {

namespace {

using namespace scan;

constexpr int kThreads = 128;
constexpr int kTile = 8;

template <int L>
struct Geo {
  static constexpr int SP = 4 * L;                           // states with padding
  static constexpr int kChunk = 16 * L < 64 ? 16 * L : 64;   // tokens
  static constexpr int kBlock = 2 * kThreads / L;            // channels of a CTA
  static constexpr int kTiles = kChunk / kTile;
  static __host__ __device__ int per_group(int E, int G) { return (E / G + kBlock - 1) / kBlock; }
};

// What a chunk alone adds: one channel's four states a thread.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads)
scan_bwd_chunks_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  constexpr int CC = kThreads / L, SP = 4 * L, TT = 16, NE = TT / L, NB = (TT * SP + kThreads - 1) / kThreads;
  __shared__ __align__(16) float4 dus[TT][CC];  // delta, u, ds
  __shared__ __align__(16) float bm[TT][SP], cm[TT][SP];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, Eg = a.E / a.G, per = (Eg + CC - 1) / CC, blocks = a.G * per;
  const int k = blockIdx.x / blocks, blk = blockIdx.x - k * blocks, group = blk / per, c0 = (blk - group * per) * CC;
  const int b = blockIdx.y, n = tokens_of(a, b), t0 = k * pl.chunk, live = min(n, t0 + pl.chunk);
  const int ci = tid / L, s0 = tid % L * 4, e = group * Eg + min(c0 + ci, Eg - 1);
  const bool vec = a.S % 4 == 0;
  const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
  const float2 A2[2] = {make_float2(A4.x * kLog2e, A4.y * kLog2e), make_float2(A4.z * kLog2e, A4.w * kLog2e)};
  float2 h[2] = {both(0.f), both(0.f)}, P[2] = {both(1.f), both(1.f)}, g[2] = {both(0.f), both(0.f)};
  const int lc = tid % CC, lt = tid / CC, le = group * Eg + min(c0 + lc, Eg - 1);
  const bool there = c0 + lc < Eg;
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + le;
  const T *dt = reinterpret_cast<const T *>(a.dt) + b * a.sdt[0] + le;
  const T *dy = reinterpret_cast<const T *>(a.dy) + b * a.sdy[0] + le;
  const T *z = a.z ? reinterpret_cast<const T *>(a.z) + b * a.sz[0] + le : nullptr;
  const T *Bp = reinterpret_cast<const T *>(a.Bm) + b * a.sB[0] + group * a.sB[2];
  const T *Cp = reinterpret_cast<const T *>(a.Cm) + b * a.sC[0] + group * a.sC[2];
  const float bias = a.bias ? a.bias[le] : 0.f;
  float dsum = 0.f;
  for (int t = t0; t < live; t += TT) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int at = t + lt + i * L;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (there && at < live) {
        v.x = to_float(dt[at * a.sdt[1]]) + bias;
        if (a.softplus) v.x = softplus(v.x);
        v.y = v.x * to_float(x[at * a.sx[1]]);
        v.z = to_float(dy[at * a.sdy[1]]);
        if (z) v.z *= silu(to_float(z[at * a.sz[1]]));
      }
      dsum += v.x;
      dus[lt + i * L][lc] = v;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int j = tid + i * kThreads, at = t + j / SP, s = j % SP;
      if (j < TT * SP) {
        const bool in = at < live && s < a.S;
        (&bm[0][0])[j] = in ? to_float(Bp[at * a.sB[1] + s]) : 0.f;
        (&cm[0][0])[j] = in ? to_float(Cp[at * a.sC[1] + s]) : 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const float4 v = dus[j][ci];
      const float4 B4 = *reinterpret_cast<const float4 *>(&bm[j][s0]), C4 = *reinterpret_cast<const float4 *>(&cm[j][s0]);
      const float2 Bv[2] = {make_float2(B4.x, B4.y), make_float2(B4.z, B4.w)};
      const float2 Cv[2] = {make_float2(C4.x, C4.y), make_float2(C4.z, C4.w)};
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 w = tc::mul2(both(v.x), A2[p]), d = make_float2(ex2(w.x), ex2(w.y));
        h[p] = tc::fma2(d, h[p], tc::mul2(both(v.y), Bv[p]));
        P[p] = tc::mul2(P[p], d);
        g[p] = tc::fma2(P[p], tc::mul2(both(v.z), Cv[p]), g[p]);
      }
    }
  }
  const size_t at = ((size_t)k * a.B + b) * a.E;
  if (c0 + ci < Eg) {
    store_states(ws + (at + e) * a.S, s0, a.S, vec, make_float4(h[0].x, h[0].y, h[1].x, h[1].y));
    store_states(ws + pl.g + (at + e) * a.S, s0, a.S, vec, make_float4(g[0].x, g[0].y, g[1].x, g[1].y));
  }
  __syncthreads();
  float *red = reinterpret_cast<float *>(&dus[0][0]);
  red[lt * CC + lc] = dsum;
  __syncthreads();
  if (tid < CC && there) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < L; ++i) s += red[i * CC + tid];
    ws[pl.sum + at + le] = s;
  }
}

// The state before each chunk (y = 0) and the gradient that arrives behind it
// (y = 1), in the places of what the chunks add; also dh_in.
__global__ void __launch_bounds__(256)
scan_bwd_carry_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  pdl_launch_dependents();
  pdl_wait();
  const long long n = (long long)a.B * a.E * a.S, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const long long be = i / a.S;
  const int e = (int)(be % a.E), s = (int)(i - be * a.S);
  const float A2 = a.A[(size_t)e * a.S + s] * kLog2e;
  const float *sum = ws + pl.sum + be;
  const long long step = (long long)a.B * a.E;
  if (blockIdx.y == 0) {
    float v = a.h_in ? a.h_in[i] : 0.f;
    float *at = ws + i;
    for (int k = 0; k < pl.chunks; ++k) {
      const float l = at[k * n], w = ex2(sum[k * step] * A2);
      at[k * n] = v;
      v = fmaf(w, v, l);
    }
  } else {
    float v = a.dh_out ? a.dh_out[i] : 0.f;
    float *at = ws + pl.g + i;
    for (int k = pl.chunks - 1; k >= 0; --k) {
      const float l = at[k * n], w = ex2(sum[k * step] * A2);
      at[k * n] = v;
      v = fmaf(w, v, l);
    }
    if (a.dh_in) a.dh_in[i] = v;
  }
}

template <typename T, int L>
struct BwdSmem {
  using G = Geo<L>;
  static constexpr int kD = 0;                                     // delta [chunk][block]
  static constexpr int kU = kD + G::kChunk * G::kBlock;            // u
  static constexpr int kDs = kU + G::kChunk * G::kBlock;           // ds
  static constexpr int kB = kDs + G::kChunk * G::kBlock;           // B [chunk][SP]
  static constexpr int kC = kB + G::kChunk * G::SP;                // C
  static constexpr int kStart = kC + G::kChunk * G::SP;            // [tiles][2][threads] float4
  static constexpr int kSums = kStart + G::kTiles * 2 * kThreads * 4;  // [2][3][tile][block]: s, q, r
  static constexpr int kBc = kSums + 2 * 3 * kTile * G::kBlock;    // [2][warps][tile][2][SP]
  static constexpr int kFloats = kBc + 2 * (kThreads / 32) * kTile * 2 * G::SP;
};

template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 2)
scan_bwd_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  using G = Geo<L>;
  using M = BwdSmem<T, L>;
  constexpr int CC = G::kBlock, SP = G::SP, TC = G::kChunk;
  extern __shared__ __align__(16) float sm[];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Eg = a.E / a.G;
  const int per = G::per_group(a.E, a.G), blocks = a.G * per;
  const int k = blockIdx.x / blocks, blk = blockIdx.x - k * blocks, group = blk / per, c0 = (blk - group * per) * CC;
  const int b = blockIdx.y, n = tokens_of(a, b), t0 = k * TC, live = min(n, t0 + TC), t1 = min(a.N, t0 + TC);
  const size_t bk = (size_t)k * a.B + b;

  // ---- delta, u, ds, B and C of the chunk (zeros past the sequence's end)
  for (int j = tid; j < TC * CC; j += kThreads) {
    const int at = t0 + j / CC, c = j % CC;
    float d = 0.f, u = 0.f, ds = 0.f;
    if (c0 + c < Eg && at < live) {
      const int e = group * Eg + c0 + c;
      d = to_float(reinterpret_cast<const T *>(a.dt)[b * a.sdt[0] + at * a.sdt[1] + e]) + (a.bias ? a.bias[e] : 0.f);
      if (a.softplus) d = softplus(d);
      u = d * to_float(reinterpret_cast<const T *>(a.x)[b * a.sx[0] + at * a.sx[1] + e]);
      ds = to_float(reinterpret_cast<const T *>(a.dy)[b * a.sdy[0] + at * a.sdy[1] + e]);
      if (a.z) ds *= silu(to_float(reinterpret_cast<const T *>(a.z)[b * a.sz[0] + at * a.sz[1] + e]));
    }
    sm[M::kD + j] = d;
    sm[M::kU + j] = u;
    sm[M::kDs + j] = ds;
  }
  for (int j = tid; j < TC * SP; j += kThreads) {
    const int at = t0 + j / SP, s = j % SP;
    const bool in = at < live && s < a.S;
    sm[M::kB + j] = in ? to_float(reinterpret_cast<const T *>(a.Bm)[b * a.sB[0] + at * a.sB[1] + group * a.sB[2] + s]) : 0.f;
    sm[M::kC + j] = in ? to_float(reinterpret_cast<const T *>(a.Cm)[b * a.sC[0] + at * a.sC[1] + group * a.sC[2] + s]) : 0.f;
  }

  // ---- four states of channels ca, ca + 1
  const int s0 = lane % L * 4, ca = tid / L * 2;
  const bool vec = a.S % 4 == 0;
  float2 A2[2][2], h[2][2], ag[2][2], dA[2][2];
  bool own[2];
  int ech[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    own[c] = c0 + ca + c < Eg;
    const int e = ech[c] = group * Eg + min(c0 + ca + c, Eg - 1);
    const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
    // (0 for a channel that is not there: it takes part in the sums over channels)
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 h4 = own[c] ? load_states(ws + (bk * a.E + e) * a.S, s0, a.S, vec) : none;
    const float4 g4 = own[c] ? load_states(ws + pl.g + (bk * a.E + e) * a.S, s0, a.S, vec) : none;
    A2[c][0] = make_float2(A4.x * kLog2e, A4.y * kLog2e);
    A2[c][1] = make_float2(A4.z * kLog2e, A4.w * kLog2e);
    h[c][0] = make_float2(h4.x, h4.y);
    h[c][1] = make_float2(h4.z, h4.w);
    ag[c][0] = make_float2(g4.x, g4.y);
    ag[c][1] = make_float2(g4.z, g4.w);
    dA[c][0] = dA[c][1] = both(0.f);
  }
  __syncthreads();
  auto pairs = [&](int base, int t, float2 (&v)[2]) {
    const float4 f = *reinterpret_cast<const float4 *>(&sm[base + t * SP + s0]);
    v[0] = make_float2(f.x, f.y);
    v[1] = make_float2(f.z, f.w);
  };
  auto chans = [&](int base, int t) { return *reinterpret_cast<const float2 *>(&sm[base + t * CC + ca]); };
  float4 *start = reinterpret_cast<float4 *>(sm + M::kStart);

  // ---- forwards: the state before every tile
  const int tiles = live > t0 ? (live - t0 + kTile - 1) / kTile : 0;
  for (int i = 0; i < tiles; ++i) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      start[(i * 2 + c) * kThreads + tid] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
    if (i + 1 == tiles) break;
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int t = i * kTile + j;
      float2 B[2];
      pairs(M::kB, t, B);
      const float2 d = chans(M::kD, t), u = chans(M::kU, t);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float2 w = tc::mul2(both(c ? d.y : d.x), A2[c][p]);
          h[c][p] = tc::fma2(make_float2(ex2(w.x), ex2(w.y)), h[c][p], tc::mul2(both(c ? u.y : u.x), B[p]));
        }
    }
  }

  // ---- backwards, tile by tile
  constexpr int kChans = CC > kThreads ? CC / kThreads : 1;  // of a thread in the outputs' pass
  float sD[kChans], sBias[kChans];
#pragma unroll
  for (int i = 0; i < kChans; ++i) sD[i] = sBias[i] = 0.f;
  for (int i = tiles - 1, buf = 0; i >= 0; --i, buf ^= 1) {
    float2 dec[kTile][2][2], hs[kTile][2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float4 f = start[(i * 2 + c) * kThreads + tid];
      h[c][0] = make_float2(f.x, f.y);
      h[c][1] = make_float2(f.z, f.w);
    }
    float *sums = sm + M::kSums + buf * 3 * kTile * CC;
    float *bcp = sm + M::kBc + (buf * (kThreads / 32) + warp) * kTile * 2 * SP;
    // What a lane got of the sums of 8 values v = j * 2 + c (tokens j, channels c).
    auto put_sums = [&](float *to, int j0, float (&v)[8]) {
      share_sums<8, L>(v);
      constexpr int W = L < 8 ? L : 8;
      if (lane % L < W)
#pragma unroll
        for (int m = 0; m < 8 / W; ++m) {
          const int idx = lane % L * (8 / W) + m;
          to[(j0 + idx / 2) * CC + ca + idx % 2] = v[m];
        }
    };
    // The same for sums over the warp's channels of values v = j * 4 + s.
    auto put_bc = [&](int which, int j0, float (&v)[8]) {
      share_sums<8, 32 / L, L>(v);
      constexpr int W = 32 / L < 8 ? 32 / L : 8;
      if (lane / L < W)
#pragma unroll
        for (int m = 0; m < 8 / W; ++m) {
          const int idx = lane / L * (8 / W) + m;
          bcp[((j0 + idx / 4) * 2 + which) * SP + s0 + idx % 4] = v[m];
        }
    };
#pragma unroll
    for (int j0 = 0; j0 < kTile; j0 += 4) {
      float sv[8], cv[8];
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const int t = i * kTile + j;
        float2 B[2], C[2];
        pairs(M::kB, t, B);
        pairs(M::kC, t, C);
        const float2 d = chans(M::kD, t), u = chans(M::kU, t), ds = chans(M::kDs, t);
        float2 dc[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 s = both(0.f);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 w = tc::mul2(both(c ? d.y : d.x), A2[c][p]);
            dec[j][c][p] = make_float2(ex2(w.x), ex2(w.y));
            hs[j][c][p] = h[c][p];
            h[c][p] = tc::fma2(dec[j][c][p], h[c][p], tc::mul2(both(c ? u.y : u.x), B[p]));
            s = p ? tc::fma2(h[c][p], C[p], s) : tc::mul2(h[c][p], C[p]);
            dc[p] = c ? tc::fma2(both(ds.y), h[c][p], dc[p]) : tc::mul2(both(ds.x), h[c][p]);
          }
          sv[(j - j0) * 2 + c] = s.x + s.y;
        }
        const int o = (j & 1) * 4;
        cv[o] = dc[0].x; cv[o + 1] = dc[0].y; cv[o + 2] = dc[1].x; cv[o + 3] = dc[1].y;
        if (j & 1) put_bc(1, j - 1, cv);
      }
      put_sums(sums, j0, sv);
    }
#pragma unroll
    for (int j0 = kTile - 4; j0 >= 0; j0 -= 4) {
      float qv[8], rv[8], bv[8];
#pragma unroll
      for (int j = j0 + 3; j >= j0; --j) {
        const int t = i * kTile + j;
        float2 B[2], C[2];
        pairs(M::kB, t, B);
        pairs(M::kC, t, C);
        const float2 d = chans(M::kD, t), u = chans(M::kU, t), ds = chans(M::kDs, t);
        float2 db[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 q = both(0.f), r = both(0.f);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 g = tc::fma2(both(c ? ds.y : ds.x), C[p], ag[c][p]);
            ag[c][p] = tc::mul2(dec[j][c][p], g);
            const float2 gp = tc::mul2(ag[c][p], hs[j][c][p]);  // g e^(delta A) h_before
            q = p ? tc::fma2(g, B[p], q) : tc::mul2(g, B[p]);
            r = p ? tc::fma2(gp, A2[c][p], r) : tc::mul2(gp, A2[c][p]);
            dA[c][p] = tc::fma2(both(c ? d.y : d.x), gp, dA[c][p]);
            db[p] = c ? tc::fma2(both(u.y), g, db[p]) : tc::mul2(both(u.x), g);
          }
          qv[(j - j0) * 2 + c] = q.x + q.y;
          rv[(j - j0) * 2 + c] = r.x + r.y;
        }
        const int o = (j & 1) * 4;
        bv[o] = db[0].x; bv[o + 1] = db[0].y; bv[o + 2] = db[1].x; bv[o + 3] = db[1].y;
        if (!(j & 1)) put_bc(0, j, bv);
      }
      put_sums(sums + kTile * CC, j0, qv);
      put_sums(sums + 2 * kTile * CC, j0, rv);
    }
    __syncthreads();
    // the channels' outputs
#pragma unroll
    for (int m = 0; m < kTile * CC / kThreads; ++m) {
      const int j = tid + m * kThreads, c = j % CC, tt = i * kTile + j / CC, at = t0 + tt;
      if (c0 + c < Eg && at < live) {
        const int e = group * Eg + c0 + c;
        const float xv = to_float(reinterpret_cast<const T *>(a.x)[b * a.sx[0] + at * a.sx[1] + e]);
        const float d = sm[M::kD + tt * CC + c], ds = sm[M::kDs + tt * CC + c];
        const float s = sums[j], q = sums[kTile * CC + j], r = sums[2 * kTile * CC + j];
        const float Dv = a.D ? a.D[e] : 0.f;
        float ddt = fmaf(xv, q, r * 0.6931471805599453f);
        if (a.softplus)
          ddt *= sigmoid(to_float(reinterpret_cast<const T *>(a.dt)[b * a.sdt[0] + at * a.sdt[1] + e]) + (a.bias ? a.bias[e] : 0.f));
        reinterpret_cast<T *>(a.dx)[b * a.sdx[0] + at * a.sdx[1] + e] = from_float<T>(fmaf(d, q, Dv * ds));
        reinterpret_cast<T *>(a.ddt)[b * a.sddt[0] + at * a.sddt[1] + e] = from_float<T>(ddt);
        if (a.z) {
          const float zv = to_float(reinterpret_cast<const T *>(a.z)[b * a.sz[0] + at * a.sz[1] + e]);
          const float dyv = to_float(reinterpret_cast<const T *>(a.dy)[b * a.sdy[0] + at * a.sdy[1] + e]);
          const float sg = sigmoid(zv);
          reinterpret_cast<T *>(a.dz)[b * a.sdz[0] + at * a.sdz[1] + e] =
              from_float<T>(dyv * fmaf(Dv, xv, s) * sg * fmaf(zv, 1.f - sg, 1.f));
        }
        sD[m % kChans] = fmaf(ds, xv, sD[m % kChans]);
        sBias[m % kChans] += ddt;
      }
    }
    // this block's share of dB and dC
    for (int j = tid; j < kTile * 2 * SP; j += kThreads) {
      const int s = j % SP, w = j / SP % 2, at = t0 + i * kTile + j / (2 * SP);
      const float *p = sm + M::kBc + buf * (kThreads / 32) * kTile * 2 * SP + j;
      float v = 0.f;
#pragma unroll
      for (int m = 0; m < kThreads / 32; ++m) v += p[m * kTile * 2 * SP];
      if (s < a.S && at < live)
        ws[pl.bc + ((((size_t)(blk - group * per) * a.B + b) * a.N + at) * a.G + group) * 2 * a.S + w * a.S + s] = v;
    }
  }
  // ---- rows past the sequence's end
  for (int j = tid; j < (t1 - max(live, t0)) * CC; j += kThreads) {
    const int at = max(live, t0) + j / CC, c = j % CC;
    if (c0 + c < Eg) {
      const int e = group * Eg + c0 + c;
      reinterpret_cast<T *>(a.dx)[b * a.sdx[0] + at * a.sdx[1] + e] = from_float<T>(0.f);
      reinterpret_cast<T *>(a.ddt)[b * a.sddt[0] + at * a.sddt[1] + e] = from_float<T>(0.f);
      if (a.z) reinterpret_cast<T *>(a.dz)[b * a.sdz[0] + at * a.sdz[1] + e] = from_float<T>(0.f);
    }
  }
  for (int j = tid; j < (t1 - max(live, t0)) * 2 * a.S; j += kThreads) {
    const int at = max(live, t0) + j / (2 * a.S);
    ws[pl.bc + ((((size_t)(blk - group * per) * a.B + b) * a.N + at) * a.G + group) * 2 * a.S + j % (2 * a.S)] = 0.f;
  }
  // ---- the chunk's sums of dA, dD and dbias
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (own[c])
      store_states(ws + (bk * a.E + ech[c]) * a.S, s0, a.S, vec, make_float4(dA[c][0].x, dA[c][0].y, dA[c][1].x, dA[c][1].y));
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kChans; ++i) {
    sm[(i * kThreads + tid) * 2] = sD[i];
    sm[(i * kThreads + tid) * 2 + 1] = sBias[i];
  }
  __syncthreads();
  for (int c = tid; c < CC; c += kThreads)
    if (c0 + c < Eg) {
      const int e = group * Eg + c0 + c;
      float v0 = 0.f, v1 = 0.f;
      // (threads c, c + CC, .. had this channel; with CC > kThreads one had it alone)
      for (int j = c; j < kThreads * kChans; j += CC) {
        v0 += sm[j * 2];
        v1 += sm[j * 2 + 1];
      }
      ws[pl.dd + bk * a.E + e] = v0;
      ws[pl.dd + ((size_t)pl.chunks * a.B + bk) * a.E + e] = v1;
    }
}

// dB, dC = the blocks' shares added in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256)
scan_bwd_bc_kernel(const ScanArgs a, const ScanBwdPlan pl, const float *__restrict__ ws) {
  pdl_launch_dependents();
  pdl_wait();
  const long long cols = (long long)a.B * a.N * a.G * 2 * a.S, c = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float v = 0.f;
  for (int i = 0; i < pl.blocks; ++i) v += ws[pl.bc + i * cols + c];
  const long long row = c / (2 * a.S);
  const int j = (int)(c - row * 2 * a.S);
  T *out = reinterpret_cast<T *>(j < a.S ? a.dBm : a.dCm);
  out[row * a.S + (j < a.S ? j : j - a.S)] = from_float<T>(v);
}

template <typename F>
cudaError_t by_lanes(int S, F f) {
  if (S <= 4) return f(std::integral_constant<int, 1>());
  if (S <= 8) return f(std::integral_constant<int, 2>());
  if (S <= 16) return f(std::integral_constant<int, 4>());
  if (S <= 32) return f(std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 16>());
}

}  // namespace

ScanBwdPlan scan_bwd_plan(const ScanArgs &a) {
  ScanBwdPlan pl;
  by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    pl.chunk = Geo<L>::kChunk;
    pl.blocks = Geo<L>::per_group(a.E, a.G);
    return cudaSuccess;
  });
  pl.chunks = (a.N + pl.chunk - 1) / pl.chunk;
  const size_t be = (size_t)a.B * a.E, st = pl.chunks * be * a.S;
  auto up = [](size_t n) { return (n + 63) / 64 * 64; };  // (16-byte vectors)
  pl.g = up(st);
  pl.sum = pl.g + up(st);
  pl.dd = pl.sum + up(pl.chunks * be);
  pl.bc = pl.dd + up(2 * pl.chunks * be);
  pl.total = pl.bc + (size_t)pl.blocks * a.B * a.N * a.G * 2 * a.S;
  return pl;
}

cudaError_t launch_scan_bwd_chunks(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value, CC = kThreads / L;
    const int blocks = a.G * ((a.E / a.G + CC - 1) / CC);
    const dim3 grid((unsigned)blocks * pl.chunks, a.B);
    return bf16 ? launch_k(scan_bwd_chunks_kernel<__nv_bfloat16, L>, grid, dim3(kThreads), 0, st, true, a, pl, ws)
                : launch_k(scan_bwd_chunks_kernel<float, L>, grid, dim3(kThreads), 0, st, true, a, pl, ws);
  });
}

cudaError_t launch_scan_bwd_carry(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  const long long n = (long long)a.B * a.E * a.S;
  return launch_k(scan_bwd_carry_kernel, dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, st, true, a, pl, ws);
}

template <typename T, int L>
static cudaError_t bwd_with(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  static std::atomic<unsigned> done{0};
  auto kern = scan_bwd_kernel<T, L>;
  const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.G * pl.blocks) * pl.chunks, a.B);
  return launch_k(kern, grid, dim3(kThreads), BwdSmem<T, L>::kFloats * sizeof(float), st, true, a, pl, ws);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    return bf16 ? bwd_with<__nv_bfloat16, L>(a, pl, ws, st) : bwd_with<float, L>(a, pl, ws, st);
  });
}

cudaError_t launch_scan_bwd_bc(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, const float *ws, cudaStream_t st) {
  const long long cols = (long long)a.B * a.N * a.G * 2 * a.S;
  const dim3 grid((unsigned)((cols + 255) / 256));
  return bf16 ? launch_k(scan_bwd_bc_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, true, a, pl, ws)
              : launch_k(scan_bwd_bc_kernel<float>, grid, dim3(256), 0, st, true, a, pl, ws);
}

}  // namespace ret
