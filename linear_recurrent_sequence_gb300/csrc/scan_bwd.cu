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
// its own CTA: forwards once, keeping the state at every 4th token, then tile
// by tile backwards with 4 tokens' decays and states in registers (running a
// state backwards instead would divide by decays that underflow).
// A thread has four states of two neighbouring channels; sums over a channel's
// states are shared out over its L lanes, sums over channels over the others.
#include <algorithm>

#include "scan.cuh"

namespace ret {

namespace {

using namespace scan;

constexpr int kMain = 128;   // threads of the chunk's CTA
constexpr int kTile = 4;

template <int L>
struct Geo {
  static constexpr int SP = 4 * L;                           // states with padding
  static constexpr int kChunk = L <= 4 ? 8 * L : 32;         // tokens
  static constexpr int kBlock = 2 * kMain / L;               // channels of a CTA
  static constexpr int kTiles = kChunk / kTile;
  static __host__ __device__ int per_group(int E, int G) { return (E / G + kBlock - 1) / kBlock; }
};

// The state before each chunk (y = 0) and the gradient that arrives behind it
// (y = 1), in the places of what the chunks add; also dh_in.  Sixteen chunks'
// values are read before any of them is replaced.  Bound by memory: four passes
// over the chunks' states (2 x 4096 x 4096 x 16: 62 us, 4.3 TB/s).
__global__ void __launch_bounds__(256)
scan_bwd_carry_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int U = 16;
  const long long n = (long long)a.B * a.E * a.S, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const long long be = i / a.S;
  const int e = (int)(be % a.E), s = (int)(i - be * a.S);
  const float A2 = a.A[(size_t)e * a.S + s] * kLog2e;
  const float *sum = ws + pl.sum + be;
  const long long step = (long long)a.B * a.E;
  const bool back = blockIdx.y != 0;
  float *at = ws + (back ? pl.g : 0) + i;
  const float *from = back ? a.dh_out : a.h_in;
  float v = from ? from[i] : 0.f;
  for (int k0 = 0; k0 < pl.chunks; k0 += U) {
    float l[U], w[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = back ? pl.chunks - 1 - k0 - j : k0 + j;
      const bool in = k0 + j < pl.chunks;
      l[j] = in ? at[k * n] : 0.f;
      w[j] = in ? sum[k * step] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = back ? pl.chunks - 1 - k0 - j : k0 + j;
      if (k0 + j < pl.chunks) {
        at[k * n] = v;
        v = fmaf(ex2(w[j] * A2), v, l[j]);
      }
    }
  }
  if (back && a.dh_in) a.dh_in[i] = v;
}

// delta, u, ds, B and C of a chunk's tokens for a block of channels.
template <typename T, int L>
struct ChunkIn {
  using G = Geo<L>;
  float d[G::kChunk][G::kBlock], u[G::kChunk][G::kBlock], ds[G::kChunk][G::kBlock];
  __align__(16) T b[G::kChunk][G::SP];
  __align__(16) T c[G::kChunk][G::SP];
};

// Where a CTA stands: chunk k of block c0 of a group's channels, sequence b.
template <int L>
struct Place {
  int k, group, block, c0, b, t0, live, t1;
  __device__ __forceinline__ Place(const ScanArgs &a) {
    using G = Geo<L>;
    const int per = G::per_group(a.E, a.G), blocks = a.G * per;
    k = blockIdx.x / blocks;
    const int blk = blockIdx.x - k * blocks;
    group = blk / per;
    block = blk - group * per;
    c0 = block * G::kBlock;
    b = blockIdx.y;
    t0 = k * G::kChunk;
    live = min(tokens_of(a, b), t0 + G::kChunk);
    t1 = min(a.N, t0 + G::kChunk);
  }
};

// A thread's four neighbouring channels as loader of their tokens (and writer of
// their gradients): every kStep-th token of the chunk.
template <typename T, int L, bool kVec>
struct Quad {
  using G = Geo<L>;
  static constexpr int QC = G::kBlock / 4, kStep = kMain / QC, kCount = G::kChunk / kStep, kAtOnce = kCount < 4 ? kCount : 4;
  int c, t, there, e;  // first channel in the block, first token, channels that are there, first channel
  const T *x, *dt, *dy, *z;
  float bias[4];
  __device__ __forceinline__ Quad(const ScanArgs &a, const Place<L> &at) {
    const int Eg = a.E / a.G;
    c = threadIdx.x % QC * 4;
    t = threadIdx.x / QC;
    there = min(4, max(0, Eg - at.c0 - c));
    e = at.group * Eg + min(at.c0 + c, Eg - 1);
    x = reinterpret_cast<const T *>(a.x) + at.b * a.sx[0] + e;
    dt = reinterpret_cast<const T *>(a.dt) + at.b * a.sdt[0] + e;
    dy = reinterpret_cast<const T *>(a.dy) + at.b * a.sdy[0] + e;
    z = a.z ? reinterpret_cast<const T *>(a.z) + at.b * a.sz[0] + e : nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = a.bias && i < there ? a.bias[e + i] : 0.f;
  }
  // All of the chunk into shared memory (zeros past the sequence's end).
  __device__ __forceinline__ void stage(const ScanArgs &a, const Place<L> &at, ChunkIn<T, L> &in) const {
#pragma unroll 1
    for (int j0 = 0; j0 < kCount; j0 += kAtOnce) {
      Four<T> xr[kAtOnce], dr[kAtOnce], yr[kAtOnce], zr[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int tok = at.t0 + t + (j0 + j) * kStep, m = tok < at.live ? there : 0;
        xr[j] = load_four<T, kVec>(x + tok * a.sx[1], m);
        dr[j] = load_four<T, kVec>(dt + tok * a.sdt[1], m);
        yr[j] = load_four<T, kVec>(dy + tok * a.sdy[1], m);
        zr[j] = load_four<T, kVec>(z + tok * a.sz[1], z ? m : 0);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int to = t + (j0 + j) * kStep;
        const bool there_t = at.t0 + to < at.live;
        float d[4], u[4], ds[4];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          float2 dv = make_float2(to_float(dr[j].v[i]) + bias[i], to_float(dr[j].v[i + 1]) + bias[i + 1]);
          if (a.softplus) dv = softplus2(dv);
          d[i] = there_t && i < there ? dv.x : 0.f;
          d[i + 1] = there_t && i + 1 < there ? dv.y : 0.f;
          u[i] = d[i] * to_float(xr[j].v[i]);
          u[i + 1] = d[i + 1] * to_float(xr[j].v[i + 1]);
          float2 g = make_float2(to_float(yr[j].v[i]), to_float(yr[j].v[i + 1]));
          if (z) g = tc::mul2(g, silu2(make_float2(to_float(zr[j].v[i]), to_float(zr[j].v[i + 1]))));
          ds[i] = g.x;
          ds[i + 1] = g.y;
        }
        *reinterpret_cast<float4 *>(&in.d[to][c]) = make_float4(d[0], d[1], d[2], d[3]);
        *reinterpret_cast<float4 *>(&in.u[to][c]) = make_float4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<float4 *>(&in.ds[to][c]) = make_float4(ds[0], ds[1], ds[2], ds[3]);
      }
    }
    const T *Bp = reinterpret_cast<const T *>(a.Bm) + at.b * a.sB[0] + at.group * a.sB[2];
    const T *Cp = reinterpret_cast<const T *>(a.Cm) + at.b * a.sC[0] + at.group * a.sC[2];
    constexpr int kValues = G::kChunk * G::SP;
#pragma unroll
    for (int j = 0; j < (kValues + kMain - 1) / kMain; ++j) {
      const int o = threadIdx.x + j * kMain, tok = at.t0 + o / G::SP, s = o % G::SP;
      if (kValues % kMain && o >= kValues) break;
      const bool there_t = tok < at.live && s < a.S;
      (&in.b[0][0])[o] = there_t ? Bp[tok * a.sB[1] + s] : from_float<T>(0.f);
      (&in.c[0][0])[o] = there_t ? Cp[tok * a.sC[1] + s] : from_float<T>(0.f);
    }
  }
};

// A thread's four states of two neighbouring channels: A log2(e), and the
// operands of its tokens.
template <typename T, int L>
struct Duo {
  int s0, ca, e[2];  // first state, first channel in the block, channels
  bool own[2], vec;
  float2 A2[2][2];   // [channel][pair of states]
  __device__ __forceinline__ Duo(const ScanArgs &a, const Place<L> &at) {
    const int Eg = a.E / a.G;
    s0 = threadIdx.x % L * 4;
    ca = threadIdx.x / L * 2;
    vec = a.S % 4 == 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      own[c] = at.c0 + ca + c < Eg;
      e[c] = at.group * Eg + min(at.c0 + ca + c, Eg - 1);
      const float4 A4 = load_states(a.A + (size_t)e[c] * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
      A2[c][0] = make_float2(A4.x * kLog2e, A4.y * kLog2e);
      A2[c][1] = make_float2(A4.z * kLog2e, A4.w * kLog2e);
    }
  }
  // (0 for a channel that is not there: it takes part in the sums over channels)
  __device__ __forceinline__ void load(const ScanArgs &a, const float *states, int c, float2 (&v)[2]) const {
    const float4 f = own[c] ? load_states(states + (size_t)e[c] * a.S, s0, a.S, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = make_float2(f.x, f.y);
    v[1] = make_float2(f.z, f.w);
  }
  __device__ __forceinline__ void store(const ScanArgs &a, float *states, int c, const float2 (&v)[2]) const {
    if (own[c]) store_states(states + (size_t)e[c] * a.S, s0, a.S, vec, make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
  }
  __device__ __forceinline__ float2 chans(const float *row) const { return *reinterpret_cast<const float2 *>(row + ca); }
  __device__ __forceinline__ Four<T> states(const T *row) const { return load_four<T, true>(row + s0, 4); }
};

template <typename T>
__device__ __forceinline__ float2 pair_of(const Four<T> &f, int p) {
  return make_float2(to_float(f.v[2 * p]), to_float(f.v[2 * p + 1]));
}
__device__ __forceinline__ float2 twice(const float2 &v, int c) { return both(c ? v.y : v.x); }
__device__ __forceinline__ float2 decay(float2 w) { return make_float2(ex2(w.x), ex2(w.y)); }

// What each chunk alone adds to the state after it and to the gradient before it.
// Many small CTAs: one's loads arrive while the others walk.  2 x 4096 x 4096 x 16
// bf16: 212 us, bound by packed arithmetic and exponentials (2.7 instructions a
// clock); on the forward's walk, one channel a lane, 257.
template <typename T, int L, bool kVec>
__global__ void __launch_bounds__(kMain, 5)
scan_bwd_chunks_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  using G = Geo<L>;
  extern __shared__ __align__(16) uint8_t dyn[];
  ChunkIn<T, L> &in = *reinterpret_cast<ChunkIn<T, L> *>(dyn);
  pdl_wait();
  const Place<L> at(a);
  Quad<T, L, kVec>(a, at).stage(a, at, in);
  const Duo<T, L> me(a, at);
  float2 h[2][2], P[2][2], g[2][2], sum = both(0.f);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      h[c][p] = g[c][p] = both(0.f);
      P[c][p] = both(1.f);
    }
  __syncthreads();
  for (int t = 0; t < at.live - at.t0; t += 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Four<T> Br = me.states(in.b[t + j]), Cr = me.states(in.c[t + j]);
      const float2 d = me.chans(in.d[t + j]), u = me.chans(in.u[t + j]), ds = me.chans(in.ds[t + j]);
      sum = tc::add2(sum, d);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 B = pair_of(Br, p), C = pair_of(Cr, p);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 w = decay(tc::mul2(twice(d, c), me.A2[c][p]));
          h[c][p] = tc::fma2(w, h[c][p], tc::mul2(twice(u, c), B));
          P[c][p] = tc::mul2(P[c][p], w);
          g[c][p] = tc::fma2(P[c][p], tc::mul2(twice(ds, c), C), g[c][p]);
        }
      }
    }
  }
  pdl_launch_dependents();
  const size_t bk = ((size_t)at.k * a.B + at.b) * a.E;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    me.store(a, ws + bk * a.S, c, h[c]);
    me.store(a, ws + pl.g + bk * a.S, c, g[c]);
    if (me.own[c] && me.s0 == 0) ws[pl.sum + bk + me.e[c]] = c ? sum.y : sum.x;
  }
}

template <typename T, int L>
struct MainSmem {
  using G = Geo<L>;
  ChunkIn<T, L> in;
  // A warp's states before a tile (two channels a lane), and in their place, once
  // the tile is done, its sums: [C h, g B, g p A log2(e)][token][channel].
  static constexpr int kWarpChans = 64 / L, kRegion = 3 * kTile * kWarpChans > 256 ? 3 * kTile * kWarpChans : 256;
  __align__(16) float tile[G::kTiles][kMain / 32][kRegion];
  float bc[kMain / 32][G::kChunk][2][G::SP];   // a warp's share of dB and dC
};

// One chunk of a block of channels.  2 x 4096 x 4096 x 16 bf16: 638 us, bound by
// issue slots (62% at three warps a scheduler; 476 lane-instructions a token and
// channel, about 140 of them in the sums over lanes).  A tile is as long as its
// operands, decays and states fit the registers, so that each is read once, before
// the tile's first store (a store to shared memory holds back the loads behind it;
// tiles of 8 tokens, whose operands were read for each direction, took 883 us), and
// the warps go through the tiles each by itself (with the outputs written tile by
// tile, two barriers each, 861).
template <typename T, int L, bool kVec>
__global__ void __launch_bounds__(kMain, sizeof(T) == 2 && L <= 4 ? 3 : 2)
scan_bwd_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  using G = Geo<L>;
  using Q = Quad<T, L, kVec>;
  constexpr int CC = G::kBlock, SP = G::SP;
  extern __shared__ __align__(16) uint8_t dyn[];
  MainSmem<T, L> &sm = *reinterpret_cast<MainSmem<T, L> *>(dyn);
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Place<L> at(a);
  const Q quad(a, at);
  quad.stage(a, at, sm.in);
  const Duo<T, L> me(a, at);
  const int s0 = me.s0;
  const size_t bk = ((size_t)at.k * a.B + at.b) * a.E;
  float2 h[2][2], ag[2][2], dA[2][2];  // [channel][pair of states]
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    me.load(a, ws + bk * a.S, c, h[c]);
    me.load(a, ws + pl.g + bk * a.S, c, ag[c]);
    dA[c][0] = dA[c][1] = both(0.f);
  }
  __syncthreads();

  // ---- forwards: the state before every tile
  const int tiles = at.live > at.t0 ? (at.live - at.t0 + kTile - 1) / kTile : 0;
  auto starts = [&](int i, int c) { return reinterpret_cast<float4 *>(&sm.tile[i][warp][(c * 32 + lane) * 4]); };
  auto keep_start = [&](int i) {
#pragma unroll
    for (int c = 0; c < 2; ++c) *starts(i, c) = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
  };
  if (tiles > 0) keep_start(0);
  for (int i = 0; i + 1 < tiles; ++i) {
    Four<T> Br[kTile];
    float2 dv[kTile], uv[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      Br[j] = me.states(sm.in.b[i * kTile + j]);
      dv[j] = me.chans(sm.in.d[i * kTile + j]);
      uv[j] = me.chans(sm.in.u[i * kTile + j]);
    }
#pragma unroll
    for (int j = 0; j < kTile; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 B = pair_of(Br[j], p);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 w = decay(tc::mul2(twice(dv[j], c), me.A2[c][p]));
          h[c][p] = tc::fma2(w, h[c][p], tc::mul2(twice(uv[j], c), B));
        }
      }
    keep_start(i + 1);
  }

  // ---- backwards, tile by tile
  // (each warp by itself; what a lane gets of the sums of 8 values v = j * 2 + c,
  // tokens j, channels c, and of sums over the warp's channels of v = j * 4 + s)
  constexpr int WS = L < 8 ? L : 8, WB = 32 / L < 8 ? 32 / L : 8, WC = MainSmem<T, L>::kWarpChans;
  auto put_sums = [&](float *to, const float (&v)[8]) {
    if (lane % L < WS)
#pragma unroll
      for (int m = 0; m < 8 / WS; ++m) {
        const int idx = lane % L * (8 / WS) + m;
        to[idx / 2 * WC + lane / L * 2 + idx % 2] = v[m];
      }
  };
  auto put_bc = [&](int which, int t, const float (&v)[8]) {
    if (lane / L < WB)
#pragma unroll
      for (int m = 0; m < 8 / WB; ++m) {
        const int idx = lane / L * (8 / WB) + m;
        sm.bc[warp][t + idx / 4][which][s0 + idx % 4] = v[m];
      }
  };
  for (int i = tiles - 1; i >= 0; --i) {
    Four<T> Br[kTile], Cr[kTile];
    float2 dv[kTile], uv[kTile], gv[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int t = i * kTile + j;
      Br[j] = me.states(sm.in.b[t]);
      Cr[j] = me.states(sm.in.c[t]);
      dv[j] = me.chans(sm.in.d[t]);
      uv[j] = me.chans(sm.in.u[t]);
      gv[j] = me.chans(sm.in.ds[t]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float4 f = *starts(i, c);
      h[c][0] = make_float2(f.x, f.y);
      h[c][1] = make_float2(f.z, f.w);
    }
    float2 dec[kTile][2][2], hs[kTile][2][2];  // decays, and the states before each token
    float sv[8], qv[8], rv[8], cv[2][8], bv[2][8];
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      float2 sum[2], dc[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 B = pair_of(Br[j], p), C = pair_of(Cr[j], p);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          dec[j][c][p] = decay(tc::mul2(twice(dv[j], c), me.A2[c][p]));
          hs[j][c][p] = h[c][p];
          h[c][p] = tc::fma2(dec[j][c][p], h[c][p], tc::mul2(twice(uv[j], c), B));
          sum[c] = p ? tc::fma2(h[c][p], C, sum[c]) : tc::mul2(h[c][p], C);
          dc[p] = c ? tc::fma2(twice(gv[j], c), h[c][p], dc[p]) : tc::mul2(twice(gv[j], c), h[c][p]);
        }
        cv[j / 2][(j & 1) * 4 + 2 * p] = dc[p].x;
        cv[j / 2][(j & 1) * 4 + 2 * p + 1] = dc[p].y;
      }
      sv[j * 2] = sum[0].x + sum[0].y;
      sv[j * 2 + 1] = sum[1].x + sum[1].y;
      if (j & 1) share_sums<8, 32 / L, L>(cv[j / 2]);
    }
    share_sums<8, L>(sv);
#pragma unroll
    for (int j = kTile - 1; j >= 0; --j) {
      float2 q[2], r[2], db[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 B = pair_of(Br[j], p), C = pair_of(Cr[j], p);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float2 g = tc::fma2(twice(gv[j], c), C, ag[c][p]);
          ag[c][p] = tc::mul2(dec[j][c][p], g);
          const float2 gp = tc::mul2(ag[c][p], hs[j][c][p]);  // g e^(delta A) h_before
          q[c] = p ? tc::fma2(g, B, q[c]) : tc::mul2(g, B);
          r[c] = p ? tc::fma2(gp, me.A2[c][p], r[c]) : tc::mul2(gp, me.A2[c][p]);
          dA[c][p] = tc::fma2(twice(dv[j], c), gp, dA[c][p]);
          db[p] = c ? tc::fma2(twice(uv[j], c), g, db[p]) : tc::mul2(twice(uv[j], c), g);
        }
        bv[j / 2][(j & 1) * 4 + 2 * p] = db[p].x;
        bv[j / 2][(j & 1) * 4 + 2 * p + 1] = db[p].y;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qv[j * 2 + c] = q[c].x + q[c].y;
        rv[j * 2 + c] = r[c].x + r[c].y;
      }
      if (!(j & 1)) share_sums<8, 32 / L, L>(bv[j / 2]);
    }
    share_sums<8, L>(qv);
    share_sums<8, L>(rv);
    __syncwarp();  // every lane has its start
    put_sums(&sm.tile[i][warp][0], sv);
    put_sums(&sm.tile[i][warp][kTile * WC], qv);
    put_sums(&sm.tile[i][warp][2 * kTile * WC], rv);
#pragma unroll
    for (int j = 0; j < kTile / 2; ++j) {
      put_bc(0, i * kTile + j * 2, bv[j]);
      put_bc(1, i * kTile + j * 2, cv[j]);
    }
  }
  __syncthreads();

  // ---- the channels' gradients
  float sD[4] = {}, sBias[4] = {}, Dv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) Dv[i] = a.D && i < quad.there ? a.D[quad.e + i] : 0.f;
  constexpr int UQ = Q::kAtOnce, QS = Q::kStep;
  const int qc = quad.c, there = quad.there;
#pragma unroll 1
  for (int j0 = 0; j0 < Q::kCount; j0 += UQ) {
    Four<T> xr[UQ], dr[UQ], yr[UQ], zr[UQ];
#pragma unroll
    for (int j = 0; j < UQ; ++j) {
      const int tok = at.t0 + quad.t + (j0 + j) * QS, m = tok < at.live ? there : 0;
      xr[j] = load_four<T, kVec>(quad.x + tok * a.sx[1], m);
      dr[j] = load_four<T, kVec>(quad.dt + tok * a.sdt[1], a.softplus ? m : 0);
      yr[j] = load_four<T, kVec>(quad.dy + tok * a.sdy[1], a.z ? m : 0);
      zr[j] = load_four<T, kVec>(quad.z + tok * a.sz[1], a.z ? m : 0);
    }
#pragma unroll
    for (int j = 0; j < UQ; ++j) {
      const int t = quad.t + (j0 + j) * QS, tok = at.t0 + t;
      if (tok >= at.t1) continue;
      float ddx[4] = {}, ddt[4] = {}, ddz[4] = {};  // (zeros past the sequence's end)
      if (tok < at.live) {
        const float4 d4 = *reinterpret_cast<const float4 *>(&sm.in.d[t][qc]), ds4 = *reinterpret_cast<const float4 *>(&sm.in.ds[t][qc]);
        const float d[4] = {d4.x, d4.y, d4.z, d4.w}, ds[4] = {ds4.x, ds4.y, ds4.z, ds4.w};
        const float *sums = &sm.tile[t / kTile][qc / WC][t % kTile * WC + qc % WC];
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const float2 s = *reinterpret_cast<const float2 *>(sums + c), q = *reinterpret_cast<const float2 *>(sums + kTile * WC + c);
          const float2 r = *reinterpret_cast<const float2 *>(sums + 2 * kTile * WC + c);
          const float2 xv = make_float2(to_float(xr[j].v[c]), to_float(xr[j].v[c + 1]));
          const float2 dv = make_float2(d[c], d[c + 1]), g = make_float2(ds[c], ds[c + 1]), D2 = make_float2(Dv[c], Dv[c + 1]);
          float2 v = tc::fma2(xv, q, tc::mul2(r, both(0.6931471805599453f)));  // (r has A log2(e) for A)
          if (a.softplus)
            v = tc::mul2(v, sigmoid2(make_float2(to_float(dr[j].v[c]) + quad.bias[c], to_float(dr[j].v[c + 1]) + quad.bias[c + 1])));
          ddt[c] = v.x;
          ddt[c + 1] = v.y;
          v = tc::fma2(dv, q, tc::mul2(D2, g));
          ddx[c] = v.x;
          ddx[c + 1] = v.y;
          if (a.z) {
            const float2 zv = make_float2(to_float(zr[j].v[c]), to_float(zr[j].v[c + 1])), sg = sigmoid2(zv);
            const float2 yv = make_float2(to_float(yr[j].v[c]), to_float(yr[j].v[c + 1]));
            const float2 slope = tc::mul2(sg, tc::fma2(zv, make_float2(1.f - sg.x, 1.f - sg.y), both(1.f)));
            v = tc::mul2(tc::mul2(yv, tc::fma2(D2, xv, s)), slope);
            ddz[c] = v.x;
            ddz[c + 1] = v.y;
          }
          sD[c] = fmaf(g.x, xv.x, sD[c]);
          sD[c + 1] = fmaf(g.y, xv.y, sD[c + 1]);
          sBias[c] += ddt[c];
          sBias[c + 1] += ddt[c + 1];
        }
      }
      store_four<T, kVec>(reinterpret_cast<T *>(a.dx) + at.b * a.sdx[0] + tok * a.sdx[1] + quad.e, there, ddx);
      store_four<T, kVec>(reinterpret_cast<T *>(a.ddt) + at.b * a.sddt[0] + tok * a.sddt[1] + quad.e, there, ddt);
      if (a.z) store_four<T, kVec>(reinterpret_cast<T *>(a.dz) + at.b * a.sdz[0] + tok * a.sdz[1] + quad.e, there, ddz);
    }
  }
  // this block's share of dB and dC
  for (int o = tid; o < (at.t1 - at.t0) * 2 * SP; o += kMain) {
    const int s = o % SP, w = o / SP % 2, tok = at.t0 + o / (2 * SP);
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < kMain / 32; ++q) v += (&sm.bc[q][0][0][0])[o];
    if (s < a.S)
      ws[pl.bc + ((((size_t)at.block * a.B + at.b) * a.N + tok) * a.G + at.group) * 2 * a.S + w * a.S + s] = tok < at.live ? v : 0.f;
  }
  pdl_launch_dependents();
  // ---- the chunk's sums of dA, dD and dbias
  me.store(a, ws + bk * a.S, 0, dA[0]);
  me.store(a, ws + bk * a.S, 1, dA[1]);
  __syncthreads();
  float *red = &sm.in.d[0][0];  // [2][QS][CC]
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    red[quad.t * CC + qc + c] = sD[c];
    red[(QS + quad.t) * CC + qc + c] = sBias[c];
  }
  __syncthreads();
  for (int c = tid; c < CC; c += kMain)
    if (at.c0 + c < a.E / a.G) {
      const int e = at.group * (a.E / a.G) + at.c0 + c;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll 4
      for (int j = 0; j < QS; ++j) {
        v0 += red[j * CC + c];
        v1 += red[(QS + j) * CC + c];
      }
      ws[pl.dd + bk + e] = v0;
      ws[pl.dd + (size_t)pl.chunks * a.B * a.E + bk + e] = v1;
    }
}

// dB, dC = the blocks' shares added in order, rounded once (64 blocks of 2 x 4096 x
// 2 x 16 values: 21 us, 3.3 TB/s).
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

// Vectors of four channels in every tensor (outputs: that the gradients are too)?
bool vectors_ok(const ScanArgs &a, int esz, bool outputs) {
  constexpr int step = 4;
  return a.E / a.G % step == 0 && rows_on(a, a.x, a.sx, step, esz) && rows_on(a, a.dt, a.sdt, step, esz) &&
         rows_on(a, a.dy, a.sdy, step, esz) && rows_on(a, a.z, a.sz, step, esz) &&
         (!outputs || (rows_on(a, a.dx, a.sdx, step, esz) && rows_on(a, a.ddt, a.sddt, step, esz) &&
                       (!a.z || rows_on(a, a.dz, a.sdz, step, esz))));
}

template <bool kChunks, typename T, int L, bool kVec>
cudaError_t run_with(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  static std::atomic<unsigned> done{0};
  auto kern = kChunks ? scan_bwd_chunks_kernel<T, L, kVec> : scan_bwd_kernel<T, L, kVec>;
  const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.G * pl.blocks) * pl.chunks, a.B);
  const size_t smem = kChunks ? sizeof(ChunkIn<T, L>) : sizeof(MainSmem<T, L>);
  return launch_k(kern, grid, dim3(kMain), smem, st, true, a, pl, ws);
}

template <bool kChunks, typename T>
cudaError_t run_any(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  const bool vec = vectors_ok(a, sizeof(T), !kChunks);
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    return vec ? run_with<kChunks, T, L, true>(a, pl, ws, st) : run_with<kChunks, T, L, false>(a, pl, ws, st);
  });
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
  return bf16 ? run_any<true, __nv_bfloat16>(a, pl, ws, st) : run_any<true, float>(a, pl, ws, st);
}

cudaError_t launch_scan_bwd_carry(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  const long long n = (long long)a.B * a.E * a.S;
  return launch_k(scan_bwd_carry_kernel, dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, st, true, a, pl, ws);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  return bf16 ? run_any<false, __nv_bfloat16>(a, pl, ws, st) : run_any<false, float>(a, pl, ws, st);
}

cudaError_t launch_scan_bwd_bc(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, const float *ws, cudaStream_t st) {
  const long long cols = (long long)a.B * a.N * a.G * 2 * a.S;
  const dim3 grid((unsigned)((cols + 255) / 256));
  return bf16 ? launch_k(scan_bwd_bc_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, true, a, pl, ws)
              : launch_k(scan_bwd_bc_kernel<float>, grid, dim3(256), 0, st, true, a, pl, ws);
}

}  // namespace ret
