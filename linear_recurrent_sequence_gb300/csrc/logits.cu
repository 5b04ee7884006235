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
// The alternatives cost no second pass.  The running maxima of the CTA's
// threads, each over its own V / kThreads values, give a lower bound of the
// k-th largest logit: the k-th largest of them (found bit by bit with
// counting barriers).  Only the threads whose maximum reaches the bound hold
// candidates, k of them up to ties, so only their values are read again
// (from the caches), and the few that reach the bound are ranked against one
// another.
#include "launch.h"
#include "logits.cuh"

namespace ret {

namespace {

constexpr int kThreads = 512;
constexpr int kCand = 1024;  // candidates ranked at once; more take the exact search
constexpr int kUnroll = 4;

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
  unsigned long long cand[kCand];
  int count;
  int warp_total[kThreads / 32];
};

// Calls f(key, index, valid) for the values of the warp's threads in `mask`,
// one thread's values after another, spread over the lanes.
template <typename T, typename F>
__device__ __forceinline__ void each_value(const LogitRow<T> &row, unsigned mask, F f) {
  constexpr int kVec = LogitRow<T>::kVec;
  const int lane = threadIdx.x & 31, wbase = threadIdx.x & ~31;
  while (mask) {
    const int t = wbase + __ffs(mask) - 1;
    mask &= mask - 1;
    if (lane == 0 && t < row.head) f(order_key<T>(logit_of(row.p[t])), t);
    if (lane == 0 && t < row.tail)
      f(order_key<T>(logit_of(row.p[row.tail_index() + t])), row.tail_index() + t);
    for (int i = t + lane * kThreads; i < row.nvec; i += 32 * kThreads) {
      LogitVec<T> v;
      v.load(row.p + row.index(i));
      float x[kVec];
      v.get(x);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(order_key<T>(x[j]), row.index(i) + j);
    }
  }
}

// The largest b with at least k of the CTA's values of `count_ge(b)`.
template <typename T, typename C>
__device__ __forceinline__ uint32_t kth_key(int k, C count_ge) {
  uint32_t best = 0;
  for (int bit = sizeof(T) == 2 ? 15 : 31; bit >= 0; --bit) {
    const uint32_t t = best | (1u << bit);
    const int n = count_ge(t);
    if (n >= k) best = t;
    if (n == k) break;
  }
  return best;
}

// Fills sh.cand with the (key, ~index) pairs of the row's k largest values
// and at most kCand in all; returns their number (fewer than k only where
// the row has fewer values above -infinity).  own: this thread's maximum.
template <typename T>
__device__ int top_candidates(const LogitRow<T> &row, float own, int k, TopShared &sh) {
  const uint32_t mine = order_key<T>(own), masked = order_key<T>(-INFINITY);
  uint32_t bound = kth_key<T>(k, [&](uint32_t t) { return __syncthreads_count(mine >= t); });
  // At least one above the masked values.
  bound = max(bound, masked + 1);
  auto push = [&](uint32_t key, int idx, uint32_t least) {
    if (key >= least) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kCand) sh.cand[at] = ((unsigned long long)key << 32) | (uint32_t)~idx;
    }
  };
  auto collect = [&](uint32_t least) {
    __syncthreads();
    if (threadIdx.x == 0) sh.count = 0;
    __syncthreads();
    each_value(row, __ballot_sync(0xffffffffu, mine >= least),
               [&](uint32_t key, int idx) { push(key, idx, least); });
    __syncthreads();
    return sh.count;
  };
  int n = collect(bound);
  if (n <= kCand) return n;
  // Many values reach the bound: equal ones (a mask of the type's lowest
  // value), or large ones that few threads hold.  Take the values above it,
  // if need be above the exact k-th largest, and then of the values at it
  // the first ones in index order.
  n = collect(bound + 1);
  if (n > kCand) {
    bound = kth_key<T>(k, [&](uint32_t t) {
      __syncthreads();
      if (threadIdx.x == 0) sh.count = 0;
      __syncthreads();
      int c = 0;
      each_value(row, __ballot_sync(0xffffffffu, mine >= t),
                 [&](uint32_t key, int) { c += key >= t; });
      if (c) atomicAdd(&sh.count, c);
      __syncthreads();
      return sh.count;
    });
    n = collect(bound + 1);  // fewer than k, or k where the search ended early
  }
  int need = k - n;
  constexpr int kVec = LogitRow<T>::kVec;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int tiles = (row.nvec + kThreads - 1) / kThreads;
  for (int tile = -1; tile <= tiles && need > 0; ++tile) {
    // head values, tiles of one vector a thread, tail values
    uint32_t hit = 0;
    int base = 0;
    if (tile < 0 || tile == tiles) {
      const int cnt = tile < 0 ? row.head : row.tail;
      base = (tile < 0 ? 0 : row.tail_index()) + threadIdx.x;
      hit = (int)threadIdx.x < cnt && order_key<T>(logit_of(row.p[base])) == bound;
    } else {
      const int i = tile * kThreads + threadIdx.x;
      if (i < row.nvec && mine >= bound) {
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
    for (int w = 0; w < kThreads / 32; ++w) {
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

template <typename T>
__global__ void __launch_bounds__(kThreads)
token_logprobs_kernel(const LogprobArgs a) {
  __shared__ Softmax joined[kThreads / 32];
  __shared__ TopShared sh;
  pdl_launch_dependents();
  pdl_wait();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const LogitRow<T> row(reinterpret_cast<const T *>(a.x) + row_offset(a.sx, r), a.V);
    const int tid = threadIdx.x;
    long long token = -1;
    float xt = 0.f;
    if (tid == 0 && a.tokens) {
      token = a.id64 ? reinterpret_cast<const long long *>(a.tokens)[r]
                     : (long long)reinterpret_cast<const int *>(a.tokens)[r];
      if (token >= 0 && token < a.V) xt = logit_of(row.p[token]);
    }
    Softmax acc = Softmax::none();
    for (int i = tid; i < row.nvec; i += kUnroll * kThreads) {
      LogitVec<T> v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int at = i + j * kThreads;
        if (at < row.nvec)
          v[j].load(row.p + row.index(at));
        else
          v[j].fill_masked();
      }
      acc.group<T, kUnroll, true>(v, a.scale);
    }
    if (tid < row.head) {
      const float x = logit_of(row.p[tid]);
      acc.raise(x, a.scale);
      acc.take(x, a.scale);
    }
    if (tid < row.tail) {
      const float x = logit_of(row.p[row.tail_index() + tid]);
      acc.raise(x, a.scale);
      acc.take(x, a.scale);
    }
    const Softmax all = join_cta(acc, a.scale, joined);
    const bool empty = !(all.m > -INFINITY);
    const float lnz = logf(all.s);
    if (tid == 0) {
      float lp = 0.f, ent = empty ? 0.f : lnz - 0.6931471805599453f * (all.u / all.s);
      if (token >= a.V || all.bad)
        lp = token < 0 ? 0.f : __int_as_float(0x7fffffff);
      else if (token >= 0)
        lp = empty ? -INFINITY : (xt - all.m) * a.inv_t - lnz;
      if (all.bad) ent = __int_as_float(0x7fffffff);
      if (a.logprob) a.logprob[r] = lp;
      if (a.entropy) a.entropy[r] = ent;
    }
    if (a.top > 0) {
      const int n = all.bad || empty ? 0 : top_candidates(row, acc.m, a.top, sh);
      for (int i = tid; i < n; i += kThreads) {
        const unsigned long long key = sh.cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += sh.cand[j] > key;
        if (rank < a.top) {
          const float x = key_value<T>((uint32_t)(key >> 32));
          if (a.top_logprob) a.top_logprob[r * a.top + rank] = (x - all.m) * a.inv_t - lnz;
          if (a.top_id) a.top_id[r * a.top + rank] = (long long)(uint32_t)~(uint32_t)key;
        }
      }
      for (int i = n + tid; i < a.top; i += kThreads) {
        if (a.top_logprob)
          a.top_logprob[r * a.top + i] = all.bad ? __int_as_float(0x7fffffff) : -INFINITY;
        if (a.top_id) a.top_id[r * a.top + i] = -1;
      }
    }
    __syncthreads();  // the shared lists of this row have been read
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, int bf16, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const dim3 grid((unsigned)(a.rows < (1LL << 30) ? a.rows : (1LL << 30)));
  return bf16 ? launch_k(token_logprobs_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, true, a)
              : launch_k(token_logprobs_kernel<float>, grid, dim3(kThreads), 0, st, true, a);
}

}  // namespace ret
