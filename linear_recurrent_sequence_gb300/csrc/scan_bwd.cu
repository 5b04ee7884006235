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

constexpr int kMain = 128;   // threads of the chunk's CTA
constexpr int kTile = 8;

template <int L>
struct Geo {
  static constexpr int SP = 4 * L;                           // states with padding
  static constexpr int kChunk = 16 * L < 64 ? 16 * L : 64;   // tokens: two tiles of the first pass
  static constexpr int kBlock = 2 * kMain / L;               // channels of a CTA
  static constexpr int kTiles = kChunk / kTile;
  static_assert(kChunk == 2 * Block<L>::kTile, "a chunk is two tiles of the first pass");
  static constexpr bool kTwice = L < 16;                     // B and C twice in shared memory, as pairs
  static __host__ __device__ int per_group(int E, int G) { return (E / G + kBlock - 1) / kBlock; }
};

// The state before each chunk (y = 0) and the gradient that arrives behind it
// (y = 1), in the places of what the chunks add; also dh_in.  Eight chunks'
// values are read before any of them is replaced.
__global__ void __launch_bounds__(256)
scan_bwd_carry_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int U = 8;
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

template <int L>
struct MainSmem {
  using G = Geo<L>;
  float d[G::kChunk][G::kBlock], u[G::kChunk][G::kBlock], ds[G::kChunk][G::kBlock];  // delta, u, ds
  float b[G::kChunk][G::SP * (G::kTwice ? 2 : 1)], c[G::kChunk][G::SP * (G::kTwice ? 2 : 1)];
  float4 start[G::kTiles][2][kMain];           // the state before a tile: channel 0, 1
  float sums[3][kTile][G::kBlock];             // sum C h, sum g B, sum g p A log2(e)
  float bc[kMain / 32][kTile][2][G::SP];       // a warp's share of dB and dC
};

// One chunk of a block of channels.  f32x2 pairs are the thread's two channels:
// delta, u and ds come as pairs out of shared memory, B and C are kept there
// twice each (but for S > 32, where that would leave room for one CTA an SM).
template <typename T, int L, bool kVec>
__global__ void __launch_bounds__(kMain, 2)
scan_bwd_kernel(const ScanArgs a, const ScanBwdPlan pl, float *__restrict__ ws) {
  using G = Geo<L>;
  constexpr int CC = G::kBlock, SP = G::SP, TC = G::kChunk, QC = CC / 4;  // quads of channels
  extern __shared__ __align__(16) uint8_t dyn[];
  MainSmem<L> &sm = *reinterpret_cast<MainSmem<L> *>(dyn);
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Eg = a.E / a.G;
  const int per = G::per_group(a.E, a.G), blocks = a.G * per;
  const int k = blockIdx.x / blocks, blk = blockIdx.x - k * blocks, group = blk / per, c0 = (blk - group * per) * CC;
  const int b = blockIdx.y, n = tokens_of(a, b), t0 = k * TC, live = min(n, t0 + TC), t1 = min(a.N, t0 + TC);
  const size_t bk = (size_t)k * a.B + b;

  // ---- a quad of channels, as loader of their tokens and writer of their gradients
  const int qc = tid % QC * 4, qt = tid / QC;  // channel in the block, first token
  constexpr int QS = kMain / QC;               // tokens between a thread's
  const int there = min(4, max(0, Eg - c0 - qc)), qe = group * Eg + min(c0 + qc, Eg - 1);
  const T *x = reinterpret_cast<const T *>(a.x) + b * a.sx[0] + qe;
  const T *dt = reinterpret_cast<const T *>(a.dt) + b * a.sdt[0] + qe;
  const T *dy = reinterpret_cast<const T *>(a.dy) + b * a.sdy[0] + qe;
  const T *z = a.z ? reinterpret_cast<const T *>(a.z) + b * a.sz[0] + qe : nullptr;
  float bias[4], Dv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bias[i] = a.bias && i < there ? a.bias[qe + i] : 0.f;
    Dv[i] = a.D && i < there ? a.D[qe + i] : 0.f;
  }

  // delta, u, ds, B and C of the chunk (zeros past the sequence's end)
  constexpr int NQ = TC / QS, UQ = NQ < 4 ? NQ : 4;  // quads a thread, of which at once
#pragma unroll 1
  for (int j0 = 0; j0 < NQ; j0 += UQ) {
    Four<T> xr[UQ], dr[UQ], yr[UQ], zr[UQ];
#pragma unroll
    for (int j = 0; j < UQ; ++j) {
      const int at = t0 + qt + (j0 + j) * QS, m = at < live ? there : 0;
      xr[j] = load_four<T, kVec>(x + at * a.sx[1], m);
      dr[j] = load_four<T, kVec>(dt + at * a.sdt[1], m);
      yr[j] = load_four<T, kVec>(dy + at * a.sdy[1], m);
      zr[j] = load_four<T, kVec>(z + at * a.sz[1], z ? m : 0);
    }
#pragma unroll
    for (int j = 0; j < UQ; ++j) {
      const int t = qt + (j0 + j) * QS;
      float d[4], u[4], ds[4];
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float2 dv = make_float2(to_float(dr[j].v[i]) + bias[i], to_float(dr[j].v[i + 1]) + bias[i + 1]);
        if (a.softplus) dv = softplus2(dv);
        const bool in = t0 + t < live;
        d[i] = in && i < there ? dv.x : 0.f;
        d[i + 1] = in && i + 1 < there ? dv.y : 0.f;
        u[i] = d[i] * to_float(xr[j].v[i]);
        u[i + 1] = d[i + 1] * to_float(xr[j].v[i + 1]);
        float2 g = make_float2(to_float(yr[j].v[i]), to_float(yr[j].v[i + 1]));
        if (z) g = tc::mul2(g, silu2(make_float2(to_float(zr[j].v[i]), to_float(zr[j].v[i + 1]))));
        ds[i] = g.x;
        ds[i + 1] = g.y;
      }
      *reinterpret_cast<float4 *>(&sm.d[t][qc]) = make_float4(d[0], d[1], d[2], d[3]);
      *reinterpret_cast<float4 *>(&sm.u[t][qc]) = make_float4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<float4 *>(&sm.ds[t][qc]) = make_float4(ds[0], ds[1], ds[2], ds[3]);
    }
  }
  {
    const T *Bp = reinterpret_cast<const T *>(a.Bm) + b * a.sB[0] + group * a.sB[2];
    const T *Cp = reinterpret_cast<const T *>(a.Cm) + b * a.sC[0] + group * a.sC[2];
    constexpr int NB = (TC * SP + kMain - 1) / kMain;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int o = tid + j * kMain, t = o / SP, s = o % SP, at = t0 + t;
      if (NB * kMain > TC * SP && o >= TC * SP) break;
      const bool in = at < live && s < a.S;
      const float Bv = in ? to_float(Bp[at * a.sB[1] + s]) : 0.f, Cv = in ? to_float(Cp[at * a.sC[1] + s]) : 0.f;
      if (G::kTwice) {
        *reinterpret_cast<float2 *>(&sm.b[t][2 * s]) = both(Bv);
        *reinterpret_cast<float2 *>(&sm.c[t][2 * s]) = both(Cv);
      } else {
        sm.b[t][s] = Bv;
        sm.c[t][s] = Cv;
      }
    }
  }

  // ---- four states of channels ca, ca + 1
  const int s0 = lane % L * 4, ca = tid / L * 2;
  const bool vec = a.S % 4 == 0;
  float2 A2[4], h[4], ag[4], dA[4];
  bool own[2];
  int ech[2];
  {
    float A[2][4], hv[2][4], gv[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      own[c] = c0 + ca + c < Eg;
      const int e = ech[c] = group * Eg + min(c0 + ca + c, Eg - 1);
      // (0 for a channel that is not there: it takes part in the sums over channels)
      const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
      const float4 h4 = own[c] ? load_states(ws + (bk * a.E + e) * a.S, s0, a.S, vec) : none;
      const float4 g4 = own[c] ? load_states(ws + pl.g + (bk * a.E + e) * a.S, s0, a.S, vec) : none;
      A[c][0] = A4.x; A[c][1] = A4.y; A[c][2] = A4.z; A[c][3] = A4.w;
      hv[c][0] = h4.x; hv[c][1] = h4.y; hv[c][2] = h4.z; hv[c][3] = h4.w;
      gv[c][0] = g4.x; gv[c][1] = g4.y; gv[c][2] = g4.z; gv[c][3] = g4.w;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      A2[s] = make_float2(A[0][s] * kLog2e, A[1][s] * kLog2e);
      h[s] = make_float2(hv[0][s], hv[1][s]);
      ag[s] = make_float2(gv[0][s], gv[1][s]);
      dA[s] = both(0.f);
    }
  }
  __syncthreads();
  auto per_state = [&](const float *row, float2 (&v)[4]) {
    if (G::kTwice) {
      const float4 p = *reinterpret_cast<const float4 *>(row + 2 * s0), q = *reinterpret_cast<const float4 *>(row + 2 * s0 + 4);
      v[0] = make_float2(p.x, p.y);
      v[1] = make_float2(p.z, p.w);
      v[2] = make_float2(q.x, q.y);
      v[3] = make_float2(q.z, q.w);
    } else {
      const float4 p = *reinterpret_cast<const float4 *>(row + s0);
      v[0] = both(p.x);
      v[1] = both(p.y);
      v[2] = both(p.z);
      v[3] = both(p.w);
    }
  };
  auto chans = [&](const float *row) { return *reinterpret_cast<const float2 *>(row + ca); };

  // ---- forwards: the state before every tile
  const int tiles = live > t0 ? (live - t0 + kTile - 1) / kTile : 0;
  for (int i = 0; i < tiles; ++i) {
    sm.start[i][0][tid] = make_float4(h[0].x, h[1].x, h[2].x, h[3].x);
    sm.start[i][1][tid] = make_float4(h[0].y, h[1].y, h[2].y, h[3].y);
    if (i + 1 == tiles) break;
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int t = i * kTile + j;
      float2 B[4];
      per_state(sm.b[t], B);
      const float2 d = chans(sm.d[t]), u = chans(sm.u[t]);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float2 w = tc::mul2(d, A2[s]);
        h[s] = tc::fma2(make_float2(ex2(w.x), ex2(w.y)), h[s], tc::mul2(u, B[s]));
      }
    }
  }

  // ---- backwards, tile by tile
  float sD[4] = {}, sBias[4] = {};
  constexpr int NW = kTile / QS > 0 ? kTile / QS : 1;  // quads of a tile a thread writes
  // What a lane gets of the sums of 8 values v = j * 2 + c (tokens j, channels c),
  // and of sums over the warp's channels of values v = j * 4 + s.  (Held back to
  // the tile's end they would cost more in spilled registers than the loads that
  // a store holds back: 1226 us for 883.)
  auto put_sums = [&](float (*to)[CC], int j0, float (&v)[8]) {
    share_sums<8, L>(v);
    constexpr int W = L < 8 ? L : 8;
    if (lane % L < W)
#pragma unroll
      for (int m = 0; m < 8 / W; ++m) {
        const int idx = lane % L * (8 / W) + m;
        to[j0 + idx / 2][ca + idx % 2] = v[m];
      }
  };
  auto put_bc = [&](int which, int j0, float (&v)[8]) {
    share_sums<8, 32 / L, L>(v);
    constexpr int W = 32 / L < 8 ? 32 / L : 8;
    if (lane / L < W)
#pragma unroll
      for (int m = 0; m < 8 / W; ++m) {
        const int idx = lane / L * (8 / W) + m;
        sm.bc[warp][j0 + idx / 4][which][s0 + idx % 4] = v[m];
      }
  };
  for (int i = tiles - 1; i >= 0; --i) {
    // (the channels' rows for the outputs, on their way meanwhile)
    Four<T> xr[NW], dr[NW], yr[NW], zr[NW];
    const bool writes = QS <= kTile || qt < kTile;
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      const int at = t0 + i * kTile + qt + m * QS, c = writes && at < live ? there : 0;
      xr[m] = load_four<T, kVec>(x + at * a.sx[1], c);
      dr[m] = load_four<T, kVec>(dt + at * a.sdt[1], a.softplus ? c : 0);
      yr[m] = load_four<T, kVec>(dy + at * a.sdy[1], z ? c : 0);
      zr[m] = load_four<T, kVec>(z + at * a.sz[1], z ? c : 0);
    }
    float2 dec[kTile][4], hs[kTile][4];  // decays, and the states before each token
    {
      const float4 p = sm.start[i][0][tid], q = sm.start[i][1][tid];
      h[0] = make_float2(p.x, q.x);
      h[1] = make_float2(p.y, q.y);
      h[2] = make_float2(p.z, q.z);
      h[3] = make_float2(p.w, q.w);
    }
#pragma unroll
    for (int j0 = 0; j0 < kTile; j0 += 4) {
      float sv[8], cv[8];
#pragma unroll
      for (int j = j0; j < j0 + 4; ++j) {
        const int t = i * kTile + j;
        float2 B[4], C[4];
        per_state(sm.b[t], B);
        per_state(sm.c[t], C);
        const float2 d = chans(sm.d[t]), u = chans(sm.u[t]), ds = chans(sm.ds[t]);
        float2 sum = both(0.f);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float2 w = tc::mul2(d, A2[s]);
          dec[j][s] = make_float2(ex2(w.x), ex2(w.y));
          hs[j][s] = h[s];
          h[s] = tc::fma2(dec[j][s], h[s], tc::mul2(u, B[s]));
          sum = s ? tc::fma2(h[s], C[s], sum) : tc::mul2(h[s], C[s]);
          const float2 dc = tc::mul2(ds, h[s]);
          cv[(j & 1) * 4 + s] = dc.x + dc.y;
        }
        sv[(j - j0) * 2] = sum.x;
        sv[(j - j0) * 2 + 1] = sum.y;
        if (j & 1) put_bc(1, j - 1, cv);
      }
      put_sums(sm.sums[0], j0, sv);
    }
#pragma unroll
    for (int j0 = kTile - 4; j0 >= 0; j0 -= 4) {
      float qv[8], rv[8], bv[8];
#pragma unroll
      for (int j = j0 + 3; j >= j0; --j) {
        const int t = i * kTile + j;
        float2 B[4], C[4];
        per_state(sm.b[t], B);
        per_state(sm.c[t], C);
        const float2 d = chans(sm.d[t]), u = chans(sm.u[t]), ds = chans(sm.ds[t]);
        float2 q = both(0.f), r = both(0.f);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float2 g = tc::fma2(ds, C[s], ag[s]);
          ag[s] = tc::mul2(dec[j][s], g);
          const float2 gp = tc::mul2(ag[s], hs[j][s]);  // g e^(delta A) h_before
          q = s ? tc::fma2(g, B[s], q) : tc::mul2(g, B[s]);
          r = s ? tc::fma2(gp, A2[s], r) : tc::mul2(gp, A2[s]);
          dA[s] = tc::fma2(d, gp, dA[s]);
          const float2 db = tc::mul2(u, g);
          bv[(j & 1) * 4 + s] = db.x + db.y;
        }
        qv[(j - j0) * 2] = q.x;
        qv[(j - j0) * 2 + 1] = q.y;
        rv[(j - j0) * 2] = r.x;
        rv[(j - j0) * 2 + 1] = r.y;
        if (!(j & 1)) put_bc(0, j, bv);
      }
      put_sums(sm.sums[1], j0, qv);
      put_sums(sm.sums[2], j0, rv);
    }
    __syncthreads();
    // the channels' gradients
#pragma unroll
    for (int m = 0; m < NW; ++m) {
      const int j = qt + m * QS, at = t0 + i * kTile + j;
      if (writes && at < live) {
        float ddx[4], ddt[4], ddz[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float xv = to_float(xr[m].v[c]), d = sm.d[i * kTile + j][qc + c], ds = sm.ds[i * kTile + j][qc + c];
          const float s = sm.sums[0][j][qc + c], q = sm.sums[1][j][qc + c], r = sm.sums[2][j][qc + c];
          ddt[c] = fmaf(xv, q, r * 0.6931471805599453f);  // (r has A log2(e) for A)
          if (a.softplus) ddt[c] *= sigmoid(to_float(dr[m].v[c]) + bias[c]);
          ddx[c] = fmaf(d, q, Dv[c] * ds);
          if (z) {
            const float zv = to_float(zr[m].v[c]), sg = sigmoid(zv);
            ddz[c] = to_float(yr[m].v[c]) * fmaf(Dv[c], xv, s) * sg * fmaf(zv, 1.f - sg, 1.f);
          }
          if (c < there) {
            sD[c] = fmaf(ds, xv, sD[c]);
            sBias[c] += ddt[c];
          }
        }
        store_four<T, kVec>(reinterpret_cast<T *>(a.dx) + b * a.sdx[0] + at * a.sdx[1] + qe, there, ddx);
        store_four<T, kVec>(reinterpret_cast<T *>(a.ddt) + b * a.sddt[0] + at * a.sddt[1] + qe, there, ddt);
        if (z) store_four<T, kVec>(reinterpret_cast<T *>(a.dz) + b * a.sdz[0] + at * a.sdz[1] + qe, there, ddz);
      }
    }
    // this block's share of dB and dC
#pragma unroll
    for (int m = 0; m < (kTile * 2 * SP + kMain - 1) / kMain; ++m) {
      const int o = tid + m * kMain;
      if (o < kTile * 2 * SP) {
        const int s = o % SP, w = o / SP % 2, at = t0 + i * kTile + o / (2 * SP);
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < kMain / 32; ++q) v += (&sm.bc[q][0][0][0])[o];
        if (s < a.S && at < live)
          ws[pl.bc + ((((size_t)(blk - group * per) * a.B + b) * a.N + at) * a.G + group) * 2 * a.S + w * a.S + s] = v;
      }
    }
    __syncthreads();
  }
  pdl_launch_dependents();
  // ---- rows past the sequence's end
  const int end = max(live, t0);
  const float zero[4] = {};
  for (int at = end + qt; at < t1; at += QS) {
    store_four<T, kVec>(reinterpret_cast<T *>(a.dx) + b * a.sdx[0] + at * a.sdx[1] + qe, there, zero);
    store_four<T, kVec>(reinterpret_cast<T *>(a.ddt) + b * a.sddt[0] + at * a.sddt[1] + qe, there, zero);
    if (z) store_four<T, kVec>(reinterpret_cast<T *>(a.dz) + b * a.sdz[0] + at * a.sdz[1] + qe, there, zero);
  }
  for (int j = tid; j < (t1 - end) * 2 * a.S; j += kMain) {
    const int at = end + j / (2 * a.S);
    ws[pl.bc + ((((size_t)(blk - group * per) * a.B + b) * a.N + at) * a.G + group) * 2 * a.S + j % (2 * a.S)] = 0.f;
  }
  // ---- the chunk's sums of dA, dD and dbias
  if (own[0]) store_states(ws + (bk * a.E + ech[0]) * a.S, s0, a.S, vec, make_float4(dA[0].x, dA[1].x, dA[2].x, dA[3].x));
  if (own[1]) store_states(ws + (bk * a.E + ech[1]) * a.S, s0, a.S, vec, make_float4(dA[0].y, dA[1].y, dA[2].y, dA[3].y));
  __syncthreads();
  float *red = &sm.d[0][0];  // [2][QS][CC]
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    red[qt * CC + qc + c] = sD[c];
    red[(QS + qt) * CC + qc + c] = sBias[c];
  }
  __syncthreads();
  for (int c = tid; c < CC; c += kMain)
    if (c0 + c < Eg) {
      const int e = group * Eg + c0 + c;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll 4
      for (int j = 0; j < QS; ++j) {
        v0 += red[j * CC + c];
        v1 += red[(QS + j) * CC + c];
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

// Vectors of four channels in every tensor?
bool vectors_ok(const ScanArgs &a, int esz) {
  constexpr int step = 4;
  return a.E / a.G % step == 0 && rows_on(a, a.x, a.sx, step, esz) && rows_on(a, a.dt, a.sdt, step, esz) &&
         rows_on(a, a.dy, a.sdy, step, esz) && rows_on(a, a.z, a.sz, step, esz) &&
         rows_on(a, a.dx, a.sdx, step, esz) && rows_on(a, a.ddt, a.sddt, step, esz) &&
         (!a.z || rows_on(a, a.dz, a.sdz, step, esz));
}

template <typename T, int L, bool kVec>
cudaError_t main_with(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  static std::atomic<unsigned> done{0};
  auto kern = scan_bwd_kernel<T, L, kVec>;
  const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.G * pl.blocks) * pl.chunks, a.B);
  return launch_k(kern, grid, dim3(kMain), sizeof(MainSmem<L>), st, true, a, pl, ws);
}

template <typename T>
cudaError_t main_any(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  const bool vec = vectors_ok(a, sizeof(T));
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    return vec ? main_with<T, L, true>(a, pl, ws, st) : main_with<T, L, false>(a, pl, ws, st);
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

cudaError_t launch_scan_bwd_carry(const ScanArgs &a, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  const long long n = (long long)a.B * a.E * a.S;
  return launch_k(scan_bwd_carry_kernel, dim3((unsigned)((n + 255) / 256), 2), dim3(256), 0, st, true, a, pl, ws);
}

cudaError_t launch_scan_bwd(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, float *ws, cudaStream_t st) {
  return bf16 ? main_any<__nv_bfloat16>(a, pl, ws, st) : main_any<float>(a, pl, ws, st);
}

cudaError_t launch_scan_bwd_bc(const ScanArgs &a, int bf16, const ScanBwdPlan &pl, const float *ws, cudaStream_t st) {
  const long long cols = (long long)a.B * a.N * a.G * 2 * a.S;
  const dim3 grid((unsigned)((cols + 255) / 256));
  return bf16 ? launch_k(scan_bwd_bc_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, true, a, pl, ws)
              : launch_k(scan_bwd_bc_kernel<float>, grid, dim3(256), 0, st, true, a, pl, ws);
}

}  // namespace ret
