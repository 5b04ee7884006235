// Log probabilities of given tokens, entropy and the top alternatives of
// logits x [rows][V] at temperature T, in one pass over each row:
//   m = max x, z = sum e^{(x - m) / T},
//   log p_t = (x_t - m) / T - ln z,   H = ln z - sum p (x - m) / T,
// and the k largest logits, equal values by the lower index.  A logit of
// -infinity is a masked token: probability 0, never an alternative.
//
// Bound by memory: each logit is read once (2 or 4 bytes) and costs one
// exponential and about six other operations.
//
// The alternatives cost no second pass.  The maxima of the CTA's threads, each
// of its own values, give a lower bound of the k-th largest logit: the k-th
// largest of them, which one warp finds by bisection.  Only the threads whose
// maximum reaches the bound hold candidates, k of them up to ties, so only
// their values are read again (from the caches), and the few that reach the
// bound are ranked against one another.  Where a cluster shares a row, each CTA
// finds the k largest of its slice, and ranks its own among all of them.
#include <type_traits>

#include "launch.h"
#include "logits.cuh"

namespace ret {

namespace {

constexpr int kCand = 1024;  // candidates ranked at once, and vectors that hold
constexpr int kQueue = 512;  // some; more take the exact search
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

struct TopShared {
  alignas(16) unsigned long long cand[kCand];  // in a cluster also [ctas][kMaxTop]
  unsigned long long sorted[kMaxTop];  // this CTA's, in order
  uint4 raw[kQueue];                   // vectors that hold candidates
  int at[kQueue];                      // and their numbers
  uint32_t own[kRowThreads];
  uint32_t bound;
  int count, queued, listed;
  int warp_total[kRowWarps];
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

// Fills sh.cand with the (key, ~index) pairs of the slice's k largest values
// and at most kCand in all; returns their number (fewer than k only where
// the slice has fewer values above -infinity).  own: this thread's maximum.
template <typename T>
__device__ int top_candidates(const LogitRow<T> &row, const RowSlice &slice, int single, float own,
                              int k, TopShared &sh) {
  const uint32_t mine = order_key<T>(own), masked = order_key<T>(-INFINITY);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  sh.own[threadIdx.x] = mine;
  if (threadIdx.x == 0) sh.count = sh.queued = 0;
  __syncthreads();
  if (wid == 0) {
    uint32_t q[kRowWarps], lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int i = 0; i < kRowWarps; ++i) {
      q[i] = sh.own[lane + 32 * i];
      lo = min(lo, q[i]);
      hi = max(hi, q[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t b = kth_key(lo, hi, k, [&](uint32_t t) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < kRowWarps; ++i) c += q[i] >= t;
      return __reduce_add_sync(0xffffffffu, c);
    });
    if (lane == 0) sh.bound = max(b, masked + 1);  // masked values are no candidates
  }
  __syncthreads();
  uint32_t bound = sh.bound;
  auto push = [&](float x, int idx) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCand) sh.cand[at] = ((unsigned long long)order_key<T>(x) << 32) | (uint32_t)~idx;
  };
  constexpr int kVec = LogitRow<T>::kVec;
  // The values from `least` up.  A warp goes through the values of its threads
  // that hold some, four threads at a time, and queues the vectors with some.
  auto collect = [&](uint32_t least) {
    const float value = key_value<T>(least);
    unsigned mask = __ballot_sync(0xffffffffu, mine >= least);
    const int base = slice.v0 + (threadIdx.x & ~31) + lane * kRowThreads;
    while (mask) {
      int t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t[j] = mask ? base + __ffs(mask) - 1 : slice.v1;
        mask &= mask - 1;
      }
      for (int more = t[0] - lane * kRowThreads; more < slice.v1; more += 32 * kRowThreads) {
        LogitVec<T> v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t[j] < slice.v1) v[j].load(row.p + row.index(t[j]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const LogitVec<T> one[1] = {v[j]};
          if (t[j] < slice.v1 && LogitVec<T>::max_of(one) >= value) {
            const int at = atomicAdd(&sh.queued, 1);
            if (at < kQueue) {
              sh.raw[at] = *reinterpret_cast<const uint4 *>(&v[j].raw);
              sh.at[at] = t[j];
            }
          }
          t[j] = min(t[j], slice.v1) + 32 * kRowThreads;
        }
      }
    }
    if (single >= 0) {
      const float x = logit_of(row.p[single]);
      if (x >= value) push(x, single);
    }
    __syncthreads();
    const int queued = sh.queued;
    for (int i = threadIdx.x; i < min(queued, kQueue); i += kRowThreads) {
      LogitVec<T> v;
      *reinterpret_cast<uint4 *>(&v.raw) = sh.raw[i];
      float x[kVec];
      v.get(x);
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (x[j] >= value) push(x[j], row.index(sh.at[i]) + j);
    }
    __syncthreads();
    return queued > kQueue ? kCand + 1 : sh.count;
  };
  auto restart = [&] {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = sh.queued = 0;
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
          for (int i = slice.v0 + threadIdx.x; i < slice.v1; i += kRowThreads)
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
  const int tiles = (slice.v1 - slice.v0 + kRowThreads - 1) / kRowThreads;
  for (int tile = -1; tile <= tiles && need > 0; ++tile) {
    // values before the vectors, tiles of one vector a thread, values after
    uint32_t hit = 0;
    int base = 0;
    if (tile < 0 || tile == tiles) {
      base = single;
      hit = (tile < 0 ? threadIdx.x < 8 : threadIdx.x >= 8) && single >= 0 &&
            order_key<T>(logit_of(row.p[single])) == bound;
    } else {
      const int i = slice.v0 + tile * kRowThreads + threadIdx.x;
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
    for (int w = 0; w < kRowWarps; ++w) {
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

template <typename T, bool kEntropy, bool kTop>
__global__ void __launch_bounds__(kRowThreads, 5)
token_logprobs_kernel(const LogprobArgs a) {
  __shared__ Softmax parts[kRowWarps], mine;
  __shared__ std::conditional_t<kTop, TopShared, int> shared_top;
  TopShared &sh = reinterpret_cast<TopShared &>(shared_top);  // used with kTop only
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
    WarpSoftmax acc;
    int i = slice.v0 + (tid & ~31);  // of the warp's first lane: the loops are the warp's
    for (; i + 31 + (kUnroll - 1) * kRowThreads < slice.v1; i += kUnroll * kRowThreads) {
      LogitVec<T> v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) v[j].load(row.p + row.index(i + lane + j * kRowThreads));
      acc.group<T, kUnroll, kEntropy>(v, a.scale);
    }
    if (i < slice.v1) {
      LogitVec<T> v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int at = i + lane + j * kRowThreads;
        if (at < slice.v1)
          v[j].load(row.p + row.index(at));
        else
          v[j].fill_masked();
      }
      acc.group<T, kUnroll, kEntropy>(v, a.scale);
    }
    if (tid < 32) acc.single<kEntropy>(single >= 0 ? logit_of(row.p[single]) : -INFINITY, a.scale);
    const Softmax all = join_row<kEntropy>(acc.all<kEntropy>(), a.scale, ctas, parts, &mine);
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
      const bool none = all.bad || empty;
      int n = none ? 0 : top_candidates(row, slice, single, acc.own, a.top, sh);
      auto put = [&](unsigned long long key, int at) {
        const float x = key_value<T>((uint32_t)(key >> 32));
        if (a.top_logprob) a.top_logprob[r * a.top + at] = (x - all.m) * a.inv_t - lnz;
        if (a.top_id) a.top_id[r * a.top + at] = (long long)(uint32_t)~(uint32_t)key;
      };
      for (int c = tid; c < n; c += kRowThreads) {
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
        if (tid >> 5 < (int)ctas) {
          const uint32_t c = tid >> 5;
          const int there = (int)cluster_word(&sh.listed, c);
#pragma unroll
          for (int j = 0; j < 2 * kMaxTop / 32; ++j)
            if (lane + 32 * j < 2 * there)
              reinterpret_cast<uint32_t *>(sh.cand)[2 * kMaxTop * c + lane + 32 * j] =
                  cluster_word(reinterpret_cast<const uint32_t *>(sh.sorted) + lane + 32 * j, c);
          if (lane == 0) sh.warp_total[c] = there;
        }
        __syncthreads();
        cluster_have_read();
        int total = 0;
        for (uint32_t c = 0; c < ctas; ++c) total += sh.warp_total[c];
        if (tid < n) {
          const unsigned long long key = sh.sorted[tid];
          int at = 0;  // how many of each list come before key: of its own, tid
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c >= (int)ctas) continue;
            const int there = sh.warp_total[c];
            int lo = 0;
#pragma unroll
            for (int step = kMaxTop; step > 0; step >>= 1)
              if (lo + step <= there && sh.cand[kMaxTop * c + lo + step - 1] > key) lo += step;
            at += lo;
          }
          if (at < a.top) put(key, at);
        }
        n = rank == 0 ? min(total, a.top) : a.top;
      }
      for (int c = n + tid; c < a.top; c += kRowThreads) {
        if (a.top_logprob) a.top_logprob[r * a.top + c] = all.bad ? nan_value() : -INFINITY;
        if (a.top_id) a.top_id[r * a.top + c] = -1;
      }
    }
    // the shared lists of this row have been read, by the other CTAs too
    if (ctas > 1) cluster_wait_read();
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch(const LogprobArgs &a, cudaStream_t st) {
  const int ctas = row_ctas(a.rows, (long long)a.V * sizeof(T), 1LL << 40, 4LL * device_sms());
  auto kern = a.entropy ? (a.top > 0 ? token_logprobs_kernel<T, true, true> : token_logprobs_kernel<T, true, false>)
                        : (a.top > 0 ? token_logprobs_kernel<T, false, true> : token_logprobs_kernel<T, false, false>);
  return launch_rows(kern, a.rows, ctas, kRowThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, int bf16, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  return bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace ret
