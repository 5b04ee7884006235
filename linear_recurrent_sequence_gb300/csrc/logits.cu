// Log probabilities of given tokens, entropy and the top alternatives of
// logits x [rows][V] at temperature T, in one pass over each row:
//   m = max x, z = sum e^{(x - m) / T},
//   log p_t = (x_t - m) / T - ln z,   H = ln z - sum p (x - m) / T,
// and the k largest logits, equal values by the lower index.  A logit of
// -infinity is a masked token: probability 0, never an alternative.
//
// Bound by memory: each logit is read once (2 or 4 bytes) and costs one
// exponential and about six other operations.  4096 x 65536 bf16: 85 us without
// alternatives, 6.3 TB/s, 99 us with five; fp32 2000 x 50001 74 us, 5.4 TB/s.  Few
// rows are bound by the latency of the row's steps: 8 x 131072 bf16 4.4 us, with
// 20 alternatives 10.2 us.
//
// The alternatives cost no second pass.  Split among more than k groups of the
// CTA's threads, the values have a k-th largest of the groups' maxima that is a
// lower bound of the k-th largest logit: 32 groups of neighbouring lanes for
// k <= 32 (each warp finds the bound for itself by bisection with ballots), all
// threads beyond (one warp finds it).  Only the threads whose maximum reaches
// the bound hold candidates, so only their values are read again (from the
// caches), and the few that reach the bound are ranked against one another.
// Where a cluster shares a row, each CTA finds the k largest of its slice, and
// ranks its own among all of them.
#include <type_traits>

#include "launch.h"
#include "logits.cuh"

namespace ret {

namespace {

constexpr int kCand = 1024;  // candidates ranked at once; more take the exact search
constexpr int kGroups = 32;  // of threads, for up to so many alternatives
// Threads a slice.
template <int kT>
constexpr int kWarps = kT / 32;
constexpr int kUnroll = 4;
constexpr int kMaxTop = RETNET_MAX_TOP;

// Unsigned integer that orders as the value does (-0 counts as +0).
template <typename T>
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return sizeof(T) == 2 ? k >> 16 : k;
}

template <typename T>
__device__ __forceinline__ float key_value(uint32_t k) {
  if (sizeof(T) == 2) {
    return __uint_as_float((k & 0x8000u) ? ((k & 0x7fffu) << 16) : ((~k & 0xffffu) << 16));
  }
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

template <int kT>
struct TopShared {
  alignas(16) unsigned long long cand[kCand];  // in a cluster also [ctas][kMaxTop]
  unsigned long long sorted[kMaxTop];  // this CTA's, in order
  uint32_t own[kT];                    // the threads' maxima, or the groups'
  uint32_t bound;
  int count, listed;
  int warp_total[kWarps<kT> < 8 ? 8 : kWarps<kT>];
};

// The largest b in [lo, hi] with count_ge(b) >= k, or any b with count_ge(b)
// == k (count_ge(lo) >= k is known).
template <typename C>
__device__ __forceinline__ uint32_t kth_key(uint32_t lo, uint32_t hi, int k, C count_ge) {
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const int n = count_ge(mid);
    if (n >= k)
      lo = mid;
    else
      hi = mid - 1;
    if (n == k) break;
  }
  return lo;
}

// Whether the 32 groups' maxima serve: k of them, values in all of them, and
// one CTA a row (its barriers are what they save; in a cluster their looser
// bound costs more: 8 rows of 131072, 20 alternatives, 12.5 us against 11.3, when
// this was chosen).
template <int kT>
__device__ __forceinline__ bool by_groups(const RowSlice &slice, int k) {
  return k <= kGroups && slice.first && slice.last && slice.v1 - slice.v0 >= kT;
}

// Before the barrier that joins the row: the groups' (or threads') maxima.
template <typename T, int kT>
__device__ __forceinline__ void note_maxima(const RowSlice &slice, float own, int k, TopShared<kT> &sh) {
  uint32_t key = order_key<T>(own);
  if (by_groups<kT>(slice, k)) {
    constexpr int kLanes = kT / kGroups;
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, s));
    if (threadIdx.x % kLanes == 0) sh.own[threadIdx.x / kLanes] = key;
  } else {
    sh.own[threadIdx.x] = key;
  }
  if (threadIdx.x == 0) sh.count = 0;
}

// Fills sh.cand with the (key, ~index) pairs of the slice's k largest values
// and at most kCand in all; returns their number (fewer than k only where
// the slice has fewer values above -infinity).  own: this thread's maximum;
// note_maxima() was called before the last barrier.
template <typename T, int kT>
__device__ int top_candidates(const LogitRow<T> &row, const RowSlice &slice, int single, float own,
                              int k, TopShared<kT> &sh) {
  const uint32_t mine = order_key<T>(own), masked = order_key<T>(-INFINITY);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  uint32_t bound;
  if (by_groups<kT>(slice, k)) {
    const uint32_t q = sh.own[lane];
    bound = kth_key(__reduce_min_sync(0xffffffffu, q), __reduce_max_sync(0xffffffffu, q), k,
                    [&](uint32_t t) { return __popc(__ballot_sync(0xffffffffu, q >= t)); });
  } else {
    if (wid == 0) {
      uint32_t q[kWarps<kT>], lo = 0xffffffffu, hi = 0;
#pragma unroll
      for (int i = 0; i < kWarps<kT>; ++i) {
        q[i] = sh.own[lane + 32 * i];
        lo = min(lo, q[i]);
        hi = max(hi, q[i]);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      const uint32_t b = kth_key(lo, hi, k, [&](uint32_t t) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < kWarps<kT>; ++i) c += q[i] >= t;
        return __reduce_add_sync(0xffffffffu, c);
      });
      if (lane == 0) sh.bound = b;
    }
    __syncthreads();
    bound = sh.bound;
  }
  bound = max(bound, masked + 1);  // masked values are no candidates
  auto push = [&](float x, int idx) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCand) sh.cand[at] = ((unsigned long long)order_key<T>(x) << 32) | (uint32_t)~idx;
  };
  constexpr int kVec = LogitRow<T>::kVec;
  auto push_from = [&](const LogitVec<T> &v, float value, int at) {
    const LogitVec<T> one[1] = {v};
    if (!(LogitVec<T>::max_of(one) >= value)) return;
    float x[kVec];
    v.get(x);
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (x[e] >= value) push(x[e], row.index(at) + e);
  };
  // The values from `least` up.  In a short slice each thread that holds some
  // reads its own again (4096 rows of 1000, 20 alternatives: 22 us, the other
  // way 30).  In a longer one a warp goes through the values of its threads
  // that hold some, two threads at a time.
  const bool few = slice.v1 - slice.v0 <= 2 * kUnroll * kT;
  auto collect = [&](uint32_t least) {
    const float value = key_value<T>(least);
    unsigned mask = __ballot_sync(0xffffffffu, mine >= least);
    if (few) {
      if (mine >= least)
#pragma unroll 1
        for (int i = slice.v0 + threadIdx.x; i < slice.v1; i += kUnroll * kT) {
          LogitVec<T> v[kUnroll];
#pragma unroll
          for (int j = 0; j < kUnroll; ++j)
            if (i + j * kT < slice.v1)
              v[j].load(row.p + row.index(i + j * kT));
            else
              v[j].fill_masked();
#pragma unroll
          for (int j = 0; j < kUnroll; ++j) push_from(v[j], value, i + j * kT);
        }
      mask = 0;
    }
    const int base = slice.v0 + (threadIdx.x & ~31) + lane * kT;
    while (mask) {
      int t[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        t[j] = mask ? base + __ffs(mask) - 1 : slice.v1;
        mask &= mask - 1;
      }
      for (int more = t[0] - lane * kT; more < slice.v1; more += 32 * kT) {
        LogitVec<T> v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (t[j] < slice.v1) v[j].load(row.p + row.index(t[j]));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (t[j] < slice.v1) push_from(v[j], value, t[j]);
          t[j] = min(t[j], slice.v1) + 32 * kT;
        }
      }
    }
    if (single >= 0) {
      const float x = logit_of(row.p[single]);
      if (x >= value) push(x, single);
    }
    __syncthreads();
    return sh.count;
  };
  auto restart = [&] {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
  };
  // Where too many values reach the bound, equal ones (a mask of the type's
  // lowest value) or large ones that few threads hold: take the values above
  // it, if need be above the exact k-th largest, and then of the values at it
  // the first ones in index order.
  int n = 0;
  uint32_t least = bound;
#pragma unroll 1
  for (int turn = 0;; ++turn) {
    n = collect(least);
    if (turn == 0 && n <= kCand) return n;
    if (n <= kCand) break;
    if (turn == 1)
      bound = kth_key(bound, sizeof(T) == 2 ? 0xffffu : 0xffffffffu, k, [&](uint32_t t) {
        restart();
        int c = 0;
        if (mine >= t) {
          for (int i = slice.v0 + threadIdx.x; i < slice.v1; i += kT)
#pragma unroll 1
            for (int j = 0; j < kVec; ++j) c += order_key<T>(logit_of(row.p[row.index(i) + j])) >= t;
          if (single >= 0) c += order_key<T>(logit_of(row.p[single])) >= t;
        }
        if (c) atomicAdd(&sh.count, c);
        __syncthreads();
        return sh.count;
      });
    restart();
    least = bound + 1;
  }
  int need = k - n;
  const int tiles = (slice.v1 - slice.v0 + kT - 1) / kT;
  for (int tile = -1; tile <= tiles && need > 0; ++tile) {
    // values before the vectors, tiles of one vector a thread, values after
    uint32_t hit = 0;
    int base = 0;
    if (tile < 0 || tile == tiles) {
      base = single;
      hit = (tile < 0 ? threadIdx.x < 8 : threadIdx.x >= 8) && single >= 0 &&
            order_key<T>(logit_of(row.p[single])) == bound;
    } else {
      const int i = slice.v0 + tile * kT + threadIdx.x;
      if (i < slice.v1 && mine >= bound) {
        LogitVec<T> v;
        v.load(row.p + row.index(i));
        float x[kVec];
        v.get(x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) hit |= (order_key<T>(x[j]) == bound ? 1u : 0u) << j;
        base = row.index(i);
      }
    }
    int incl = __popc(hit);
    const int c = incl;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp_total[wid] = incl;
    __syncthreads();
    int before = incl - c, total = 0;
    for (int w = 0; w < kWarps<kT>; ++w) {
      if (w < wid) before += sh.warp_total[w];
      total += sh.warp_total[w];
    }
    for (int j = 0; j < kVec && before < need; ++j)
      if (hit >> j & 1) {
        sh.cand[n + before] = ((unsigned long long)bound << 32) | (uint32_t)~(base + j);
        ++before;
      }
    const int got = min(total, need);
    n += got;
    need -= got;
  }
  __syncthreads();
  return n;
}

// Asks for the first bytes of a row (from its first 16-byte boundary) to be
// brought to L2.
template <typename T>
__device__ __forceinline__ void prefetch_row(const T *p, int V, int bytes) {
  const LogitRow<T> row(p, V);
  const int n = min(bytes, row.nvec * 16);
  if (n > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p + row.head), "r"(n) : "memory");
}

// soon: how many rows are walked over at once, 0 where the row after them is
// not to be asked for.
// (The 48 registers of 1280 threads an SM spill 8 to 100 bytes a thread where
// there are alternatives.)
template <typename T, bool kEntropy, bool kTop, int kT>
__global__ void __launch_bounds__(kT, kT == 512 ? 2 : 1280 / kT)
token_logprobs_kernel(const LogprobArgs a, int soon) {
  __shared__ Softmax parts[kWarps<kT>], mine;
  __shared__ std::conditional_t<kTop, TopShared<kT>, int> shared_top;
  TopShared<kT> &sh = reinterpret_cast<TopShared<kT> &>(shared_top);  // used with kTop only
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31;
  for (long long r = blockIdx.x / ctas; r < a.rows; r += gridDim.x / ctas) {
    const LogitRow<T> row(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), a.V);
    const RowSlice slice(row, ctas, rank);
    const int single = slice.single(row);
    long long token = -1;
    float xt = 0.f;
    if (tid == 0 && rank == 0 && a.tokens) {
      token = a.id64 ? reinterpret_cast<const long long *>(a.tokens)[r]
                     : (long long)reinterpret_cast<const int *>(a.tokens)[r];
      if (token >= 0 && token < a.V) xt = logit_of(row.p[token]);
    }
    const Scale sc(a.scale);
    WarpSoftmax acc;
    int i = slice.v0 + (tid & ~31);  // of the warp's first lane: the loops are the warp's
    for (; i + 31 + (kUnroll - 1) * kT < slice.v1; i += kUnroll * kT) {
      LogitVec<T> v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) v[j].load(row.p + row.index(i + lane + j * kT));
      acc.group<T, kUnroll, kEntropy>(v, sc);
    }
    if (i < slice.v1) {
      LogitVec<T> v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int at = i + lane + j * kT;
        if (at < slice.v1)
          v[j].load(row.p + row.index(at));
        else
          v[j].fill_masked();
      }
      acc.group<T, kUnroll, kEntropy>(v, sc);
    }
    if (tid < 32) acc.single<kEntropy>(single >= 0 ? logit_of(row.p[single]) : -INFINITY, sc);
    if (kTop) note_maxima<T, kT>(slice, acc.own, a.top, sh);
    const Softmax all = join_row<kEntropy, kWarps<kT>>(acc.all<kEntropy>(sc), a.scale, ctas, parts, &mine);
    if (ctas > 1 && !kTop) cluster_have_read();
    const bool empty = !(all.m > -INFINITY);
    const float lnz = logf(all.s);
    if (tid == 0 && rank == 0) {
      float lp = 0.f;
      if (token >= a.V || all.bad)
        lp = token < 0 ? 0.f : nan_value();
      else if (token >= 0)
        lp = empty ? -INFINITY : (xt - all.m) * a.inv_t - lnz;
      if (a.logprob) a.logprob[r] = lp;
      if (kEntropy)
        a.entropy[r] = all.bad ? nan_value() : empty ? 0.f : lnz - 0.6931471805599453f * (all.u / all.s);
    }
    if (kTop) {
      if (kT == 256 && tid == 0 && soon && r + soon < a.rows)
        prefetch_row(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r + soon), a.V, kT * kUnroll * 16);
      const bool none = all.bad || empty;
      int n = none ? 0 : top_candidates<T, kT>(row, slice, single, acc.own, a.top, sh);
      auto put = [&](unsigned long long key, int at) {
        const float x = key_value<T>((uint32_t)(key >> 32));
        if (a.top_logprob) a.top_logprob[r * a.top + at] = (x - all.m) * a.inv_t - lnz;
        if (a.top_id) a.top_id[r * a.top + at] = (long long)(uint32_t)~(uint32_t)key;
      };
      for (int c = tid; c < n; c += kT) {
        const unsigned long long key = sh.cand[c];
        int at = 0, j = 0;
        for (; j + 3 < n; j += 4) {
          const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(sh.cand + j);
          const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(sh.cand + j + 2);
          at += (p.x > key) + (p.y > key) + (q.x > key) + (q.y > key);
        }
        for (; j < n; ++j) at += sh.cand[j] > key;
        if (at >= a.top) continue;
        if (ctas == 1)
          put(key, at);
        else
          sh.sorted[at] = key;
      }
      n = min(n, a.top);
      if (ctas > 1) {
        if (tid == 0) sh.listed = n;
        cluster_sync();
        // the CTAs' lists, in order, beside one another: a warp for each
        for (uint32_t c = tid >> 5; c < ctas; c += kWarps<kT>) {
          const int there = (int)cluster_word(&sh.listed, c);
#pragma unroll
          for (int j = 0; j < 2 * kMaxTop / 32; ++j)
            if (lane + 32 * j < 2 * a.top)  // (those past its length are not looked at)
              reinterpret_cast<uint32_t *>(sh.cand)[2 * kMaxTop * c + lane + 32 * j] =
                  cluster_word(reinterpret_cast<const uint32_t *>(sh.sorted) + lane + 32 * j, c);
          if (lane == 0) sh.warp_total[c] = there;
        }
        __syncthreads();
        cluster_have_read();
        int total = 0;
        for (uint32_t c = 0; c < ctas; ++c) total += sh.warp_total[c];
        // how many of each list come before a key: a thread for each key and list
        const int first = 1 << (31 - __clz(a.top)), lists = 31 - __clz((int)ctas);  // (a power of two)
        for (int j0 = 0; j0 < n; j0 += kT >> lists) {
          const int j = j0 + (tid >> lists), c = tid & ((int)ctas - 1);
          const unsigned long long key = j < n ? sh.sorted[j] : 0;
          int at = 0;
          if (j < n) {
            const int there = sh.warp_total[c];
            for (int step = first; step > 0; step >>= 1)
              if (at + step <= there && sh.cand[kMaxTop * c + at + step - 1] > key) at += step;
          }
          for (int k = (int)ctas >> 1; k > 0; k >>= 1) at += __shfl_xor_sync(0xffffffffu, at, k);
          if (c == 0 && j < n && at < a.top) put(key, at);
        }
        n = rank == 0 ? min(total, a.top) : a.top;
      }
      for (int c = n + tid; c < a.top; c += kT) {
        if (a.top_logprob) a.top_logprob[r * a.top + c] = all.bad ? nan_value() : -INFINITY;
        if (a.top_id) a.top_id[r * a.top + c] = -1;
      }
    }
    // the shared lists of this row have been read, by the other CTAs too
    if (ctas > 1) cluster_wait_read();
    __syncthreads();
  }
}

// CTAs of kT threads a row: as many as the SMs hold at once.
template <typename T>
int ctas_of(const LogprobArgs &a, int threads) {
  return row_ctas(a.rows, (long long)a.V * sizeof(T), 1LL << 40, 1024LL / threads * device_sms());
}

template <typename T, int kT>
cudaError_t launch_as(const LogprobArgs &a, cudaStream_t st) {
  auto kern = a.entropy ? (a.top > 0 ? token_logprobs_kernel<T, true, true, kT> : token_logprobs_kernel<T, true, false, kT>)
                        : (a.top > 0 ? token_logprobs_kernel<T, false, true, kT> : token_logprobs_kernel<T, false, false, kT>);
  const int ctas = ctas_of<T>(a, kT);
  // While a CTA looks for alternatives it reads nothing: it asks for the first
  // group of loads of the row that follows those now walked over.  4096 rows of
  // 65536, bf16, 5 alternatives: 98 us, without it 104.  (Many alternatives
  // take so long that it comes too soon: 128 of them 199 and 193.)
  const int soon = ctas == 1 && a.top <= kGroups ? 1280 / kT * device_sms() : 0;
  return launch_rows(kern, a.rows, ctas, kT, 0, st, a, soon);
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, cudaStream_t st) {
  const long long bytes = (long long)a.V * sizeof(T);
  // Rows that two CTAs of 512 threads an SM hold at once: 512 threads, for
  // slices longer than one group of loads and for many alternatives.  256 rows
  // of 65536, bf16, 5 alternatives: 10.6 us, with 256 threads 15.6; 301 of 50001,
  // fp32, 128 alternatives: 21.6 and 33.9.  Where one group is the slice or
  // more rows follow, 256: 8 rows of 131072 without alternatives 4.4 us, with
  // 512 threads 6.1; 4096 of 65536 with 128 alternatives 194 and 226.
  if (a.rows <= 2 * device_sms() && (a.top > kGroups || bytes / ctas_of<T>(a, 512) > 512 * kUnroll * 16))
    return launch_as<T, 512>(a, st);
  // Short rows: half the threads, since most of their cost is the row's and not
  // the walk's.  4096 rows, bf16, 20 alternatives: V = 1000 22 us with 128
  // threads; fp32 2000 x 50001 86 us against 75 with 256.
  const bool narrow = a.top <= kGroups && bytes <= 32 * 1024;
  return narrow ? launch_as<T, 128>(a, st) : launch_as<T, 256>(a, st);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, int bf16, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace ret
