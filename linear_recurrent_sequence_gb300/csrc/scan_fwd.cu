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

// What the walk over the tokens is for: the outputs, or the states that segments
// leave behind.
enum { kOut = 0, kStates = 1 };

// A tile's rows as they were read, in a ring of kRing: kAhead tiles are on their
// way, the tile before the current one still has its outputs to be finished.
template <typename T, int L, int kMode>
struct __align__(16) Tile {
  static constexpr int kAhead = sizeof(T) == 2 ? 4 : 2, kRing = kAhead + 2;
  T x[Block<L>::kTile][Block<L>::kChannels], dt[Block<L>::kTile][Block<L>::kChannels];
  T z[kMode == kStates ? 1 : Block<L>::kTile][Block<L>::kChannels];
  T B[Block<L>::kTile][Block<L>::SP], C[kMode == kStates ? 1 : Block<L>::kTile][Block<L>::SP];
};

template <typename T, int L, int kMode>
struct WalkSmem {
  __align__(16) Tile<T, L, kMode> ring[Tile<T, L, kMode>::kRing];
  float2 du[2][Block<L>::kTile][Block<L>::kChannels];  // delta, u
  float sums[kMode == kStates ? 1 : 2][Block<L>::kTile][kScan];  // of C h over a lane's states
};

// Sums of two channels' L neighbouring values each.  Where a channel has one
// 16-byte vector, every other four lanes read their two in the other order: a
// quarter of a warp then meets each bank once.
template <int L>
__device__ __forceinline__ float2 lane_sums(const float *p) {
  if constexpr (L == 1) {
    return *reinterpret_cast<const float2 *>(p);
  } else if constexpr (L == 2) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    return make_float2(v.x + v.y, v.z + v.w);
  } else {
    const int swap = L == 4 ? (threadIdx.x >> 2) & 1 : 0;
    float s[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 t = both(0.f);
#pragma unroll
      for (int i = 0; i < L; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + (c ^ swap) * L + i);
        t = i ? tc::add2(t, tc::add2(make_float2(v.x, v.y), make_float2(v.z, v.w))) : tc::add2(make_float2(v.x, v.y), make_float2(v.z, v.w));
      }
      s[c] = t.x + t.y;
    }
    return make_float2(swap ? s[1] : s[0], swap ? s[0] : s[1]);
  }
}

// A third of the CTA's warps walks the recurrence; the others keep the ring
// filled, work out step sizes and inputs a tile ahead, and add up and finish the
// outputs of the tile before: with one sequence an SM has no more than one
// recurrence warp a scheduler, and everything else that a token needs runs beside
// it.  8192 x 4096 channels x 16 states bf16: 263 us.  Bound by issue slots (82%
// where they are busiest: 128 of 152 SMs have a CTA), 190 lane-instructions a
// token and channel; before that by shared memory, where a lane's bytes cost the
// same whether other lanes read them too: B and C stay in the tensors' type
// (16 bytes a lane for bf16, 32 for fp32), delta and u are kept once.  Loads that
// waited in registers instead of a ring had a tile's time to arrive (479 us), sums
// over the lanes by shuffles 301 us for 289, half the loaders 291 for 271.
// The next kernel is let in at the end, not at the start: its CTAs would gather on
// the SMs that have none of this grid's and stay there (1129 us a call, one among
// others, for 641 at that time).
// kAsync: every row begins on a 16-byte boundary and arrives by asynchronous
// copies; else the loaders read value by value (3 x 1001 x 1537 x 11 fp32: 49 us).
template <typename T, int L, int kMode, bool kAsync>
__global__ void __launch_bounds__(kThreads, 2)
scan_walk_kernel(const ScanArgs a, const ScanSegs seg) {
  using K = Block<L>;
  using Row = Tile<T, L, kMode>;
  constexpr int CC = K::kChannels, TT = K::kTile, SP = K::SP, kAhead = Row::kAhead, kRing = Row::kRing;
  extern __shared__ __align__(16) uint8_t dyn[];
  WalkSmem<T, L, kMode> &sm = *reinterpret_cast<WalkSmem<T, L, kMode> *>(dyn);
  pdl_wait();
  const int per = K::per_group(a.E, a.G), Eg = a.E / a.G, blocks = a.G * per;
  const int k = blockIdx.x / blocks, blk = blockIdx.x - k * blocks;  // segment; block of channels
  const int group = blk / per, c0 = (blk - group * per) * CC;        // within the group
  const int b = blockIdx.y;
  const int n = tokens_of(a, b), t0 = k * seg.len, t1 = min(a.N, t0 + seg.len), live = min(t1, n);
  const int tiles = live > t0 ? (live - t0 + TT - 1) / TT : 0;

  if (threadIdx.x < kScan) {
    // ---- four states of a channel
    const int tid = threadIdx.x, ci = tid / L, s0 = tid % L * 4;
    const bool own = c0 + ci < Eg, vec = a.S % 4 == 0;
    const int e = group * Eg + min(c0 + ci, Eg - 1);
    const float4 A4 = load_states(a.A + (size_t)e * a.S, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0);
    const float2 A2[2] = {make_float2(A4.x * kLog2e, A4.y * kLog2e), make_float2(A4.z * kLog2e, A4.w * kLog2e)};
    float2 h[2] = {both(0.f), both(0.f)};
    float sum = 0.f;
    const size_t row = ((size_t)b * a.E + e) * a.S;
    if (kMode == kOut) {
      // the state that the segments before this one leave behind
      if (a.h_in) {
        const float4 v = load_states(a.h_in + row, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0);
        h[0] = make_float2(v.x, v.y);
        h[1] = make_float2(v.z, v.w);
      }
      for (int i = 0; i < k; ++i) {
        const float2 d = both(seg.sum[((size_t)i * a.B + b) * a.E + e]);
        const float4 l = load_states(seg.loc + (size_t)i * a.B * a.E * a.S + row, s0, a.S, vec);
        const float2 w0 = tc::mul2(d, A2[0]), w1 = tc::mul2(d, A2[1]);
        h[0] = tc::fma2(make_float2(ex2(w0.x), ex2(w0.y)), h[0], make_float2(l.x, l.y));
        h[1] = tc::fma2(make_float2(ex2(w1.x), ex2(w1.y)), h[1], make_float2(l.z, l.w));
      }
    }
    __syncthreads();
    for (int i = 0, slot = 0; i < tiles; ++i, slot = slot + 1 == kRing ? 0 : slot + 1) {
      const int buf = i & 1;
      const Row &r = sm.ring[slot];
      float part = 0.f;
      // Four tokens at a time, the next four's operands on their way: a warp alone
      // on its scheduler has nothing else to do, and a store to shared memory
      // holds back the loads behind it.
      struct Ops {
        float2 v;
        Four<T> B, C;
      } ops[2][4];
      auto operands = [&](int q, Ops (&o)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[j].v = sm.du[buf][q + j][ci];
          o[j].B = load_four<T, true>(&r.B[q + j][s0], 4);
          if (kMode == kOut) o[j].C = load_four<T, true>(&r.C[q + j][s0], 4);
        }
      };
      operands(0, ops[0]);
#pragma unroll
      for (int q = 0; q < TT; q += 4) {
        const Ops(&o)[4] = ops[q / 4 & 1];
        if (q + 4 < TT) operands(q + 4, ops[(q / 4 + 1) & 1]);
        float2 d[4][2], in[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 dd = both(o[j].v.x), uu = both(o[j].v.y);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 w = tc::mul2(dd, A2[p]);
            d[j][p] = make_float2(ex2(w.x), ex2(w.y));
            in[j][p] = tc::mul2(uu, make_float2(to_float(o[j].B.v[2 * p]), to_float(o[j].B.v[2 * p + 1])));
          }
          if (kMode == kStates) part += o[j].v.x;
        }
        float yq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 s;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const float2 C = kMode == kStates ? both(0.f) : make_float2(to_float(o[j].C.v[2 * p]), to_float(o[j].C.v[2 * p + 1]));
            h[p] = tc::fma2(d[j][p], h[p], in[j][p]);
            if (kMode == kOut) s = p ? tc::fma2(h[p], C, s) : tc::mul2(h[p], C);
          }
          if (kMode == kOut) yq[j] = s.x + s.y;
        }
        // (the loaders add a channel's L lanes up)
        if (kMode == kOut)
#pragma unroll
          for (int j = 0; j < 4; ++j) sm.sums[buf][q + j][tid] = yq[j];
      }
      __syncthreads();
      sum += part;
    }
    pdl_launch_dependents();
    const float4 h4 = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    if (kMode == kStates) {
      if (own) {
        store_states(seg.loc + (size_t)k * a.B * a.E * a.S + row, s0, a.S, vec, h4);
        if (s0 == 0) seg.sum[((size_t)k * a.B + b) * a.E + e] = sum;
      }
    } else {
      if (k == seg.count - 1 && own && a.h_out)
        store_states(a.h_out + row, s0, a.S, vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0, h4);
    }
    return;
  }

  // ---- loaders; each has two channels of NP tokens of a tile
  constexpr int TS = 2 * kLoad / CC, NP = TS < TT ? TT / TS : 1;  // tokens between a thread's pairs; pairs
  const int tid = threadIdx.x - kScan, lc = tid % (CC / 2) * 2, lt = tid / (CC / 2);
  const int there = TS > TT && lt >= TT ? 0 : min(2, max(0, Eg - c0 - lc));  // channels of this pair
  const bool mine = TS <= TT || lt < TT;
  const int le = group * Eg + min(c0 + lc, Eg - 1);
  T *y = reinterpret_cast<T *>(a.y) + b * a.sy[0] + le;
  const int l1 = there > 1;
  const float2 bias = a.bias ? make_float2(a.bias[le], a.bias[le + l1]) : both(0.f);
  const float2 Dv = kMode == kOut && a.D ? make_float2(a.D[le], a.D[le + l1]) : both(0.f);
  const bool gate = kMode == kOut && a.z, pairs = kAsync || (a.E / a.G % 2 == 0 && a.pair_y);

  // A tensor's rows of the tiles on their way into the ring, `cols` values wide,
  // `width` of them there; this thread's vectors (kAsync) or values move on by a
  // tile a call.
  constexpr int V = kAsync ? 16 / sizeof(T) : 1;
  struct Rows {
    const T *p;      // this thread's first vector of the next tile
    long long step;  // elements from one row to the next
    int t, c;        // its row in the tile, its column
  };
  // (turned: by the other half of the threads, where half of them are enough)
  auto rows_of = [&](const void *from, long long first, long long stride, int cols, bool turned = false) {
    const int id = turned ? tid ^ (kLoad / 2) : tid;
    Rows r;
    r.step = stride;
    r.t = id / (cols / V);
    r.c = id % (cols / V) * V;
    r.p = reinterpret_cast<const T *>(from) + first + (t0 + r.t) * stride + r.c;
    return r;
  };
  auto fetch_rows = [&](T *to, Rows &r, auto columns, int row0, int width) {
    constexpr int cols = decltype(columns)::value, hop = kLoad / (cols / V);  // rows between a thread's
    static_assert(cols / V <= kLoad, "a row is at most one round");
    const T *p = r.p;
#pragma unroll
    for (int t = 0; t < TT; t += hop) {
      if (hop <= TT || r.t < TT) {
        const bool in = row0 + t + r.t < live && r.c < width;
        T *at = to + (t + r.t) * cols + r.c;
        if (kAsync)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(at)), "l"(in ? p : reinterpret_cast<const T *>(a.x)), "r"(in ? 16 : 0) : "memory");
        else
          *at = in ? *p : from_float<T>(0.f);
      }
      p += hop * r.step;
    }
    r.p += TT * r.step;
  };
  const long long at_block = (long long)group * Eg + c0;
  const int width = min(CC, Eg - c0);
  Rows fx = rows_of(a.x, b * a.sx[0] + at_block, a.sx[1], CC), fd = rows_of(a.dt, b * a.sdt[0] + at_block, a.sdt[1], CC, true);
  Rows fz = rows_of(a.z, b * a.sz[0] + at_block, a.sz[1], CC);
  Rows fB = rows_of(a.Bm, b * a.sB[0] + group * a.sB[2], a.sB[1], SP), fC = rows_of(a.Cm, b * a.sC[0] + group * a.sC[2], a.sC[1], SP, true);
  auto fetch = [&](int i) {
    if (i < tiles) {
      Row &r = sm.ring[i % kRing];
      const int t = t0 + i * TT;
      const std::integral_constant<int, CC> channels;
      const std::integral_constant<int, SP> states;
      fetch_rows(&r.x[0][0], fx, channels, t, width);
      fetch_rows(&r.dt[0][0], fd, channels, t, width);
      if (gate) fetch_rows(&r.z[0][0], fz, channels, t, width);
      fetch_rows(&r.B[0][0], fB, states, t, a.S);
      if (kMode == kOut) fetch_rows(&r.C[0][0], fC, states, t, a.S);
    }
    if (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto two = [&](const T(*rows)[CC], int t) { return *reinterpret_cast<const Two<T> *>(&rows[t][lc]); };
  // Tile i's rows become delta and u; past the end both are 0 and leave the state
  // as it is.
  auto put = [&](int i) {
    const int buf = i & 1, t = t0 + i * TT;
    const Row &r = sm.ring[i % kRing];
    if (!mine) return;
    const bool whole = there == 2 && t + TT <= live;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int at = lt + j * TS;
      const float2 xs = to_float2(two(r.x, at));
      float2 d = tc::add2(to_float2(two(r.dt, at)), bias);
      if (a.softplus) d = softplus2(d);
      if (!whole) {
        if (there < 1 || t + at >= live) d.x = 0.f;
        if (there < 2 || t + at >= live) d.y = 0.f;
      }
      const float2 u = tc::mul2(d, xs);
      *reinterpret_cast<float4 *>(&sm.du[buf][at][lc]) = make_float4(d.x, u.x, d.y, u.y);
    }
  };
  auto finish = [&](int i) {
    const int buf = i & 1, t = t0 + i * TT;
    const Row &r = sm.ring[i % kRing];
    T *to = y + (t + lt) * a.sy[1];
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int at = lt + j * TS;
      float2 v = tc::fma2(Dv, to_float2(two(r.x, at)), lane_sums<L>(&sm.sums[buf][at][lc * L]));
      if (gate) v = tc::mul2(v, silu2(to_float2(two(r.z, at))));
      if (t + at < t1) {
        const bool in = t + at < live;
        store_pair(to, pairs, there, in ? v.x : 0.f, in ? v.y : 0.f);
      }
      to += TS * a.sy[1];
    }
  };
  // Wait until all but the newest n tiles have arrived, then (all loaders') data is visible.
  auto arrived = [&] {
    if (kAsync) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
  };

#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) fetch(i);
  arrived();
  asm volatile("bar.sync 1, %0;" ::"n"(kLoad) : "memory");
  if (tiles > 0) put(0);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    fetch(i + kAhead);
    if (kMode == kOut && i > 0) finish(i - 1);
    if (i + 1 < tiles) put(i + 1);
    arrived();
    __syncthreads();
  }
  if (kMode == kOut && tiles > 0) finish(tiles - 1);
  pdl_launch_dependents();
  if (kMode == kOut)  // whole tiles past the sequence's end
    for (int at = t0 + tiles * TT + lt; at < t1; at += TS < TT ? TS : TT) store_pair(y + at * a.sy[1], pairs, there, 0.f, 0.f);
}

// One token.  A lane has four states of R sequences' same channel at a time and
// walks over the sequences, so that A is read once for them and the next ones'
// states are on their way; what a sequence's channel needs once (step size,
// gate, output) is shared out over the channel's lanes.  Bound by the states'
// bytes and, at 16 warps an SM, by the latency of its loads (3.9 of 7.7 cycles
// between a warp's instructions): 128 x 8192 x 16 bf16 43 us (3.3 TB/s; one CTA for
// each four sequences, without the next ones' loads, 54), fp32 50, 1 x 8192 x 16
// bf16 8 us.  Four sequences beside the next four's loads pass the 128 registers
// that two CTAs leave: 28 bytes are spilled with 16 states of bf16, 96 of fp32, 190 to
// 208 with B and C value by value; at bf16 1.3% of the instructions.
constexpr int kStepThreads = 256;

template <typename T, int R>
struct StepIn {
  float4 h[R];
  Four<T> B[R], C[R];
  T x, dt, z;
};

template <typename T, int L, int R, bool kVec>
__global__ void __launch_bounds__(kStepThreads, R == 1 ? 4 : 2)
scan_step_kernel(const ScanArgs a) {
  static_assert(R == 1 || R <= L, "a lane has one sequence at most to finish");
  pdl_wait();
  constexpr int CC = kStepThreads / L;
  const int lane = threadIdx.x & 31, ci = threadIdx.x / L, sub = threadIdx.x % L, s0 = sub * 4;
  const int c = blockIdx.x * CC + ci, e = min(c, a.E - 1), g = e / (a.E / a.G);
  const bool own = c < a.E, vec = a.S % 4 == 0;
  const bool va = vec && reinterpret_cast<uintptr_t>(a.A) % 16 == 0;
  const bool vi = vec && reinterpret_cast<uintptr_t>(a.h_in) % 16 == 0;
  const bool vo = vec && reinterpret_cast<uintptr_t>(a.h_out) % 16 == 0;
  const size_t step = (size_t)a.E * a.S, row = (size_t)e * a.S;
  auto load = [&](int b0, StepIn<T, R> &in) {
    if (b0 >= a.B) return;
    const int there = min(R, a.B - b0), mine = b0 + min(sub % R, there - 1);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < there) {
        in.h[r] = load_states(a.h_in + row + (b0 + r) * step, s0, a.S, vi);
        in.B[r] = load_four<T, kVec>(reinterpret_cast<const T *>(a.Bm) + (b0 + r) * a.sB[0] + g * a.sB[2] + s0, a.S - s0);
        in.C[r] = load_four<T, kVec>(reinterpret_cast<const T *>(a.Cm) + (b0 + r) * a.sC[0] + g * a.sC[2] + s0, a.S - s0);
      }
    in.x = reinterpret_cast<const T *>(a.x)[mine * a.sx[0] + e];
    in.dt = reinterpret_cast<const T *>(a.dt)[mine * a.sdt[0] + e];
    if (a.z) in.z = reinterpret_cast<const T *>(a.z)[mine * a.sz[0] + e];
  };
  int b0 = blockIdx.y * R;
  const int hop = gridDim.y * R;
  StepIn<T, R> in;
  load(b0, in);
  const float4 A4 = load_states(a.A + row, s0, a.S, va);
  const float2 A2[2] = {make_float2(A4.x * kLog2e, A4.y * kLog2e), make_float2(A4.z * kLog2e, A4.w * kLog2e)};
  const float bias = a.bias ? a.bias[e] : 0.f, Dv = a.D ? a.D[e] : 0.f;
  for (; b0 < a.B; b0 += hop) {
    const StepIn<T, R> now = in;
    load(b0 + hop, in);
    const int there = min(R, a.B - b0);
    const float x = to_float(now.x), gate = a.z ? silu(to_float(now.z)) : 1.f;
    float d = to_float(now.dt) + bias;
    if (a.softplus) d = softplus(d);
    const float u = d * x;
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int from = lane / L * L + r;
      const float2 dr = both(__shfl_sync(0xffffffffu, d, from)), ur = both(__shfl_sync(0xffffffffu, u, from));
      float2 h[2] = {make_float2(now.h[r].x, now.h[r].y), make_float2(now.h[r].z, now.h[r].w)}, s = both(0.f);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 w = tc::mul2(dr, A2[p]);
        const float2 B = make_float2(to_float(now.B[r].v[2 * p]), to_float(now.B[r].v[2 * p + 1]));
        h[p] = tc::fma2(make_float2(ex2(w.x), ex2(w.y)), h[p], tc::mul2(ur, B));
        s = tc::fma2(h[p], make_float2(to_float(now.C[r].v[2 * p]), to_float(now.C[r].v[2 * p + 1])), s);
      }
      sum[r] = s.x + s.y;
      if (own && r < there)
        store_states(a.h_out + row + (b0 + r) * step, s0, a.S, vo, make_float4(h[0].x, h[0].y, h[1].x, h[1].y));
    }
    share_sums<R, L>(sum);
    if (own && sub < there)
      reinterpret_cast<T *>(a.y)[(b0 + sub) * a.sy[0] + e] = from_float<T>(fmaf(Dv, x, sum[0]) * gate);
  }
  pdl_launch_dependents();
}

// Asynchronous copies of 16 bytes where every row of every tensor (and every
// block of channels, and every row of B and C) is made of whole ones.
template <typename T>
bool async_ok(const ScanArgs &a, int mode) {
  constexpr int V = 16 / sizeof(T), esz = sizeof(T);
  auto bc = [&](const void *p, const long long s[3]) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.N <= 1 || s[1] % V == 0) && (a.B <= 1 || s[0] % V == 0) &&
           (a.G <= 1 || s[2] % V == 0);
  };
  return a.E / a.G % V == 0 && a.S % V == 0 && bc(a.Bm, a.sB) && (mode == kStates || bc(a.Cm, a.sC)) &&
         rows_on(a, a.x, a.sx, V, esz) && rows_on(a, a.dt, a.sdt, V, esz) && (mode == kStates || rows_on(a, a.z, a.sz, V, esz)) &&
         (mode != kOut || a.pair_y);
}

template <typename T, int L, int kMode, bool kAsync>
cudaError_t walk_with(const ScanArgs &a, const ScanSegs &seg, cudaStream_t st) {
  static std::atomic<unsigned> done{0};
  auto kern = scan_walk_kernel<T, L, kMode, kAsync>;
  const cudaError_t e = allow_big_smem(reinterpret_cast<const void *>(kern), done);
  if (e != cudaSuccess) return e;
  // (the states of the last segment are nobody's entry)
  const int segs = kMode == kStates ? seg.count - 1 : seg.count;
  const dim3 grid((unsigned)(a.G * Block<L>::per_group(a.E, a.G)) * segs, a.B);
  return launch_k(kern, grid, dim3(kThreads), sizeof(WalkSmem<T, L, kMode>), st, true, a, seg);
}

template <typename T, int kMode>
cudaError_t walk_any(ScanArgs a, const ScanSegs &seg, cudaStream_t st) {
  a.pair_y = rows_on(a, a.y, a.sy, 2, sizeof(T));
  const bool async = async_ok<T>(a, kMode);
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value;
    if constexpr (4 * L * sizeof(T) >= 16)  // (a row of states is a vector at least)
      if (async) return walk_with<T, L, kMode, true>(a, seg, st);
    return walk_with<T, L, kMode, false>(a, seg, st);
  });
}

template <int kMode>
cudaError_t walk(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st) {
  return bf16 ? walk_any<__nv_bfloat16, kMode>(a, seg, st) : walk_any<float, kMode>(a, seg, st);
}

template <typename T, bool kMany>
cudaError_t step_any(const ScanArgs &a, cudaStream_t st) {
  auto on = [&](const void *p, const long long s[3]) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && (a.B == 1 || s[0] % 4 == 0) && (a.G == 1 || s[2] % 4 == 0);
  };
  const bool vec = a.S % 4 == 0 && on(a.Bm, a.sB) && on(a.Cm, a.sC);
  return by_lanes(a.S, [&](auto l) {
    constexpr int L = decltype(l)::value, CC = kStepThreads / L, R = !kMany ? 1 : L < 4 ? L : 4;
    // Walks over the sequences for three waves of two CTAs an SM (one wave, which
    // leaves SMs with one CTA beside others with two: 45 us for 43).
    const int nx = (a.E + CC - 1) / CC, groups = (a.B + R - 1) / R;
    const int ny = kMany ? std::min(groups, std::max(1, 6 * device_sms() / nx)) : groups;
    const dim3 grid(nx, ny);
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
  return walk<kStates>(a, bf16, seg, st);
}

cudaError_t launch_scan_fwd(const ScanArgs &a, int bf16, const ScanSegs &seg, cudaStream_t st) {
  return walk<kOut>(a, bf16, seg, st);
}

cudaError_t launch_scan_step(const ScanArgs &a, int bf16, cudaStream_t st) {
  // Walks over the sequences once one each would give every SM over 16 CTAs.
  const long long ctas = ((long long)a.E * lanes_of(a.S) + kStepThreads - 1) / kStepThreads * a.B;
  if (ctas >= 16LL * device_sms()) return bf16 ? step_any<__nv_bfloat16, true>(a, st) : step_any<float, true>(a, st);
  return bf16 ? step_any<__nv_bfloat16, false>(a, st) : step_any<float, false>(a, st);
}

}  // namespace ret
