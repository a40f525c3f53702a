// Log probabilities of given tokens, with entropy and the most probable
// alternatives, and the gradient to the logits.
//
//   m = max_j x_j,  s = sum_j exp(x_j - m)
//   logprob = x_t - m - log s
//   entropy = log s - sum_j exp(x_j - m) (x_j - m) / s
//   dx_j = [j = t] g - p_j (g + h (log p_j + entropy)),  p_j = exp(x_j - m) / s
// with g, h the gradients of the log probability and of the entropy.
//
// Forward reads the logits once.  A row is cut into segments of 256 threads x
// 8 vectors; a segment is in shared memory whole, so its maximum is known
// before its exponentials are taken and nothing is rescaled within it.  The
// segments' (m, s, t) are folded left to right.  The cut depends on the
// vocabulary alone: whether a block takes all of a row or a cluster of blocks
// shares it, the sum is the same bits, whatever the number of rows.
//
// Both directions are bound by memory where the rows are many: bf16 4096 x
// 131072 forward 195 us (5.5 TB/s, and next to the issue limit: an exponential,
// a maximum and two additions for every 2 bytes), backward 331 us (6.5 TB/s,
// the copy bandwidth being 6.69); f32 1000 x 32000 backward 42 us (6.1 TB/s),
// forward 24 us, 40 us with 8 alternatives.  The alternatives add half to the
// forward pass: a second look at the segments, and the first segment's bound.
// Rows off 16 bytes are bound by instructions backward (87 % of the issue slots)
// and by both those (64 %) and the wait for the loads forward: bf16 1000 x 50001
// 45 us where 50000 columns take 29.
//
// The alternatives are selected by the unique key (value, lower index first),
// so ties go to the lowest index and the order of work does not matter.  In a
// row's first segment each warp finds the few largest of its threads' maxima;
// the k-th largest of those of all warps bounds the k-th element from below.
// From there on only threads whose maximum reaches the bound look at their
// elements again and list what reaches it; the list is ranked at the row's end,
// or earlier when it grows, and then the bound rises.  Where ties or an order
// in the data make the list overflow, the k-th value is found by bisection.
// -inf never enters the list: what a row lacks in larger logits is filled by
// its lowest other indices.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "det_train.h"
#include "rows.cuh"

namespace det {
namespace {

typedef __nv_bfloat16 bf16;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVpt = 8;                                 // vectors of a segment per thread
// Stands for x - m where that is less, down to -inf: exp gives 0 all the same,
// and 0 times it, or times its product with a gradient, is 0.
constexpr float kLowest = -1000.f;

template <typename T>
constexpr int segment_elems() { return kThreads * kVpt * Elem<T>::kVec; }

struct Stats {
  float m, s, t;     // maximum; sum of e = exp(x - m); sum of e (x - m)
};

// The fold of two neighbouring stretches.
__device__ __forceinline__ Stats fold(const Stats& a, const Stats& b) {
  Stats r;
  r.m = max_nan(a.m, b.m);
  if (r.m == -INFINITY) return {r.m, 0.f, 0.f};
  const float da = max_nan(a.m - r.m, kLowest), db = max_nan(b.m - r.m, kLowest);
  const float ea = exp2_approx(da * kLog2e), eb = exp2_approx(db * kLog2e);
  r.s = a.s * ea + b.s * eb;
  r.t = (a.t + da * a.s) * ea + (b.t + db * b.s) * eb;
  return r;
}

// Order of float values as unsigned integers; NaN above all, -0 as +0.
__device__ __forceinline__ uint32_t order_of(float x) {
  x += 0.0f;
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  if (o == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Larger key: larger value, then lower index.
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t index) {
  return (static_cast<uint64_t>(order) << 32) | static_cast<uint64_t>(~index);
}

constexpr int kCandidates = 512;                        // of the list
constexpr int kRankAbove = 192;                         // the list is ranked when it is longer
constexpr uint32_t kAboveNegInf = 0x00800000u;          // order of the lowest value above -inf
constexpr int kMostPerWarp = 2 * kMaxTop / kWarps + 1;

// Shared state of the selection.
struct TopState {
  uint64_t cand[kCandidates];
  uint64_t list[kMaxTop];                               // ranked, descending; 0: none
  uint32_t maxima[kWarps * kMostPerWarp];
  uint32_t bound;
  int count, tally[kWarps];
};
struct NoTop {
  uint64_t list[1], cand[1];
};

// The k largest of cand[0, n) to out[0, k), descending, 0 where there are
// fewer (entries of cand that are 0 are not written).  Called by the whole
// block; out is complete after the next barrier.
__device__ __forceinline__ void rank_select(const uint64_t* cand, int n, int k, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = cand[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += cand[j] > key;
    if (rank < k && key != 0) out[rank] = key;
  }
  for (int i = n + threadIdx.x; i < k; i += kThreads) out[i] = 0;
}

// The warp's share of the maxima of its threads.
__device__ __forceinline__ int maxima_per_warp(int k) { return 2 * ((k + kWarps - 1) / kWarps) + 1; }
__device__ __forceinline__ void list_maxima(TopState& st, uint32_t own, int k) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = maxima_per_warp(k);
  uint32_t v = own;
  for (int i = 0; i < n; ++i) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, v);
    const uint32_t at = __ballot_sync(0xFFFFFFFFu, v == top);
    if (lane == __ffs(at) - 1) v = 0;
    if (lane == 0) st.maxima[warp * n + i] = top;
  }
}
// After a barrier: the k-th largest of all maxima, by the first warps; the
// bound is there after another barrier.
__device__ __forceinline__ void find_bound(TopState& st, int k) {
  const int n = kWarps * maxima_per_warp(k);
  if (static_cast<int>(threadIdx.x) < n) {
    const uint32_t v = st.maxima[threadIdx.x];
    int rank = 0;                                       // ties by place
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const uint32_t o = st.maxima[j];
      rank += o > v || (o == v && j < static_cast<int>(threadIdx.x));
    }
    if (rank == k - 1) st.bound = max(v, kAboveNegInf);
  }
}

constexpr uint32_t kOrderInf = 0xFF800000u;             // above it: NaN
// Whether f reaches the order o, whose value is `least`.
__device__ __forceinline__ bool reaches(float f, uint32_t o, float least) {
  return o > kOrderInf ? f != f : !(f < least);
}

// Lists the thread's elements of at least `bound` (slot i of r holds vector
// first + t + i * kThreads of thread t; base: index of the thread's first).
template <typename T>
__device__ __forceinline__ void list_elements(TopState& st, const uint4* r, uint32_t bound, uint32_t base) {
  constexpr int V = Elem<T>::kVec;
  const float least = value_of(bound);
  uint32_t which = 0;                                   // vectors that hold one
#pragma unroll 4
  for (int i = 0; i < kVpt; ++i) {
    float f[V];
    Elem<T>::unpack(r[i * kThreads], f);
    bool any = false;
#pragma unroll
    for (int e = 0; e < V; ++e) any |= reaches(f[e], bound, least);
    which |= static_cast<uint32_t>(any) << i;
  }
  for (; which != 0; which &= which - 1) {
    const int i = __ffs(which) - 1;
    float f[V];
    Elem<T>::unpack(r[i * kThreads], f);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (reaches(f[e], bound, least)) {
        const int at = atomicAdd(&st.count, 1);
        if (at < kCandidates)
          st.cand[at] = key_of(order_of(f[e]), base + static_cast<uint32_t>(i) * kThreads * V + e);
      }
  }
}

// The block's sum of n.
__device__ __forceinline__ int block_count(TopState& st, int n) {
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) st.tally[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) n += st.tally[w];
  return n;
}

// The list has overflowed in this segment: `held` entries of it (at most
// kRankAbove) are from before.  Leaves the k largest keys of those and of the
// segment in cand; at least k elements are known to reach `bound`.
template <typename T>
__device__ __noinline__ void top_overflow(TopState& st, const uint4* r, uint32_t base, int held, uint32_t bound,
                                          int k) {
  constexpr int V = Elem<T>::kVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t old = static_cast<int>(threadIdx.x) < held ? st.cand[threadIdx.x] : 0;
  // how many reach the order o
  auto reach = [&](uint32_t o) {
    int n = old != 0 && static_cast<uint32_t>(old >> 32) >= o;
    const float least = value_of(o);
#pragma unroll 1
    for (int i = 0; i < kVpt; ++i) {
      float f[V];
      Elem<T>::unpack(r[i * kThreads], f);
#pragma unroll
      for (int e = 0; e < V; ++e) n += reaches(f[e], o, least);
    }
    return block_count(st, n);
  };
  // the largest order that at least k reach: the bound itself where it is tied
  uint32_t kth = bound;
  if (bound != 0xFFFFFFFFu && reach(bound + 1) >= k) {
    kth = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit)
      if (reach(kth | (1u << bit)) >= k) kth |= 1u << bit;
  }
  __syncthreads();
  if (threadIdx.x == 0) st.count = 0;
  __syncthreads();
  // those above it, fewer than k; then the ties, lowest index first: the old ones (of earlier
  // segments), then group by group of vectors, thread by thread
  if (old != 0 && static_cast<uint32_t>(old >> 32) > kth) st.cand[atomicAdd(&st.count, 1)] = old;
#pragma unroll 1
  for (int i = 0; i < kVpt; ++i) {
    float f[V];
    Elem<T>::unpack(r[i * kThreads], f);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (order_of(f[e]) > kth)
        st.cand[atomicAdd(&st.count, 1)] =
            key_of(order_of(f[e]), base + static_cast<uint32_t>(i) * kThreads * V + e);
  }
  __syncthreads();
  int count = st.count;
  // (the old list is not in order: its ties are ranked among themselves)
  const bool tied = old != 0 && static_cast<uint32_t>(old >> 32) == kth;
  __syncthreads();
  uint64_t* ties = st.list;                             // (ranked anew after this)
  const int old_ties = block_count(st, tied);
  if (old_ties > 0) {
    // each round takes the largest key (lowest index) left
    uint64_t mine = tied ? old : 0;
    for (int n = 0; n < old_ties && count + n < k; ++n) {
      uint64_t best = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o);
        if (other > best) best = other;
      }
      __syncthreads();
      if (lane == 0) ties[warp] = best;
      __syncthreads();
      best = ties[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) best = ties[w] > best ? ties[w] : best;
      if (mine == best) {
        st.cand[count + n] = best;
        mine = 0;
      }
    }
    count = min(k, count + old_ties);
  }
#pragma unroll 1
  for (int i = 0; i < kVpt && count < k; ++i) {
    float f[V];
    Elem<T>::unpack(r[i * kThreads], f);
    int n = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) n += order_of(f[e]) == kth;
    // threads before this one
    int before = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int other = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += other;
    }
    __syncthreads();
    if (lane == 31) st.tally[warp] = before;
    __syncthreads();
    before -= n;
    int all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += st.tally[w];
      all += st.tally[w];
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (order_of(f[e]) == kth) {
        if (count + before < k)
          st.cand[count + before] = key_of(kth, base + static_cast<uint32_t>(i) * kThreads * V + e);
        ++before;
      }
    count = min(k, count + all);
  }
  __syncthreads();
  if (threadIdx.x == 0) st.count = count;
  __syncthreads();
}

// Entries of the list that are missing (0): -inf logits, by the row's lowest
// indices that the list does not hold.  One thread.
__device__ __forceinline__ void fill_list(uint64_t* list, int k) {
  int n = 0;
  while (n < k && list[n] != 0) ++n;
  const int held = n;
  for (uint32_t index = 0; n < k; ++index) {
    bool taken = false;
    for (int i = 0; i < held; ++i) taken |= ~static_cast<uint32_t>(list[i]) == index;
    if (!taken) list[n++] = key_of(kAboveNegInf - 1, index);
  }
}

template <typename T>
__device__ __forceinline__ float load_elem(const T* p) { return Elem<T>::to_float(*p); }

// The row's results from its folded stats and its list of alternatives.
template <typename T>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t row, const Stats& st,
                                          uint64_t* list) {
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const float log_s = logf(st.s);                       // -inf for a row of -inf alone
  if (threadIdx.x == 0) {
    a.stats[2 * row] = st.m;
    a.stats[2 * row + 1] = st.s;
    a.entropy[row] = st.s == 0.f ? 0.f : log_s - st.t / st.s;
    const int64_t t = a.tokens[row];
    float lp = 0.f;
    if (t >= a.vocab) {
      lp = __uint_as_float(0x7FC00000u);
    } else if (t >= 0) {
      lp = st.s == 0.f ? -INFINITY : (load_elem(x + t) - st.m) - log_s;
    }
    a.logprobs[row] = lp;
  }
  if (a.top > 0 && list[a.top - 1] == 0) {              // (uniform: the same word for all)
    __syncthreads();
    if (threadIdx.x == 0) fill_list(list, a.top);
    __syncthreads();
  }
  for (int i = threadIdx.x; i < a.top; i += blockDim.x) {
    const uint64_t key = list[i];
    a.top_tokens[row * a.top + i] = static_cast<int64_t>(~static_cast<uint32_t>(key));
    const float v = value_of(static_cast<uint32_t>(key >> 32));
    a.top_logprobs[row * a.top + i] = st.s == 0.f ? -INFINITY : (v - st.m) - log_s;
  }
}

// Largest and smallest of a vector's elements, NaN if one is.
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void extremes(const uint4* r, float& top, float& least, float) {
  top = -INFINITY;
  least = INFINITY;
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    float f[4];
    Elem<float>::unpack(r[i * kThreads], f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      top = max_nan(top, f[e]);
      least = min_nan(least, f[e]);
    }
  }
}
__device__ __forceinline__ void extremes(const uint4* r, float& top, float& least, bf16) {
  uint32_t hi = 0xFF80FF80u, lo = 0x7F807F80u;          // two at a time
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    const uint4 v = r[i * kThreads];
    hi = max_nan2(hi, max_nan2(max_nan2(v.x, v.y), max_nan2(v.z, v.w)));
    lo = min_nan2(lo, min_nan2(min_nan2(v.x, v.y), min_nan2(v.z, v.w)));
  }
  top = max_nan(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u));
  least = min_nan(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u));
}

// The short form of a thread's exponentials: its smallest element is at least
// kLeast, so that x log2(e) is finite, and the segment's maximum is less than
// kMostShort away from 0.  c = m log2(e) is then below 2^21 and its rounding d at
// most 2^-4; from about 2^30 on, 2^d and 2^-d would overflow.
constexpr float kLeast = -1e30f, kMostShort = 1048576.f;

constexpr int kStages = 2;                              // segments on their way or in use
constexpr int kBlocksPerSm = 3;
constexpr int kMaxSplits = 8;                           // blocks of a cluster
constexpr int kMaxPer = 8;                              // segments of a row in one of them

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(r)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ float remote_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t remote_u64(uint32_t at) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}

// A cluster of `splits` blocks takes rows cluster, cluster + clusters, ...; its
// rank r the segments r * per .. of each.  With one split the block folds its
// segments' statistics as they come; otherwise rank 0 reads every rank's from
// its shared memory and folds them in the same order (per <= kMaxPer).
template <typename T, bool kTop, bool kPlain>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    logprobs_forward_kernel(LogprobsArgs a, int segments, int per, int splits) {
  constexpr int V = Elem<T>::kVec;
  extern __shared__ uint4 ring[];
  __shared__ typename std::conditional<kTop, TopState, NoTop>::type top;
  __shared__ uint64_t joined[kTop ? kMaxTop : 1];
  __shared__ Stats seg_stats[kMaxPer], all_stats[kMaxPer * kMaxSplits];
  __shared__ float wm[2][kWarps], ws[2][kWarps], wt[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t clusters = gridDim.x / splits;
  const int seg0 = min(segments, rank * per), seg1 = min(segments, seg0 + per), own = seg1 - seg0;
  // the block's work in order: its segments of its first row, of its next, ...
  int64_t fetch_row = blockIdx.x / splits;
  int fetch_seg = seg0, fetch_stage = 0;
  uint4* slots = ring + threadIdx.x;
  auto fetch = [&]() {
    if (own > 0 && fetch_row < a.rows) {
      ring_load<T, kVpt, kPlain>(slots + fetch_stage * (kVpt * kThreads), kThreads,
                         static_cast<const T*>(a.logits) + fetch_row * a.ld, a.vocab,
                         int64_t(fetch_seg) * (kThreads * kVpt) + threadIdx.x, kThreads, Elem<T>::kNegInf);
      if (++fetch_seg == seg1) {
        fetch_seg = seg0;
        fetch_row += clusters;
      }
    }
    ring_commit();
    fetch_stage = (fetch_stage + 1) % kStages;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch();
  int stage = 0, parity = 0;
  uint32_t bound = 0;                                   // of the list's elements
  int held = 0;                                         // entries of it before the segment
  if constexpr (kTop) {
    if (threadIdx.x == 0) top.count = 0;
  }
  for (int64_t row = blockIdx.x / splits; row < a.rows; row += clusters) {
    Stats total{-INFINITY, 0.f, 0.f};
    for (int seg = seg0; seg < seg1; ++seg) {
      fetch();
      ring_wait<kStages - 1>();
      uint4* r = slots + stage * (kVpt * kThreads);
      stage = (stage + 1) % kStages;
      if (kPlain && seg == segments - 1) {              // slots past the row's end
#pragma unroll
        for (int i = 0; i < kVpt; ++i)
          if ((int64_t(seg) * (kThreads * kVpt) + threadIdx.x + i * kThreads) * V >= a.vocab)
            r[i * kThreads] = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
      }
      float best, least;
      extremes(r, best, least, T());
      const float wmax = warp_max_nan(best);
      if (lane == 0) wm[parity][warp] = wmax;
      const uint32_t own_order = kTop ? order_of(best) : 0;
      if constexpr (kTop) {
        if (seg == seg0) list_maxima(top, own_order, a.top);
      }
      __syncthreads();
      if constexpr (kTop) {
        if (seg == seg0) {
          find_bound(top, a.top);
          __syncthreads();
          bound = top.bound;
        }
      }
      float m = wm[parity][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) m = max_nan(m, wm[parity][w]);
      float s = 0.f, t = 0.f;
      if (least > kLeast && fabsf(m) < kMostShort) {
        // e = 2^(x log2 e - c) with c the rounded m log2 e; the rounding d of c
        // is a factor 2^d of every e, taken out at the end
        const float c = m * kLog2e, d = fmaf(m, kLog2e, -c);
#pragma unroll 4
        for (int i = 0; i < kVpt; ++i) {
          float f[V];
          Elem<T>::unpack(r[i * kThreads], f);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float y = fmaf(f[e], kLog2e, -c);
            const float p = exp2_approx(y);
            s += p;
            t = fmaf(p, y, t);
          }
        }
        t = 0.6931471805599453f * fmaf(-d, s, t);
        const float by = exp2_approx(-d);
        s *= by;
        t *= by;
      } else {
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 2
        for (int i = 0; i < kVpt; ++i) {
          float f[V];
          Elem<T>::unpack(r[i * kThreads], f);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float d = max_nan(f[e] - ref, kLowest);
            const float p = exp2_approx(d * kLog2e);
            s += p;
            t = fmaf(p, d, t);
          }
        }
      }
      s = warp_sum(s);
      t = warp_sum(t);
      if constexpr (kTop) {
        if (own_order >= bound)
          list_elements<T>(top, r, bound, (static_cast<uint32_t>(seg) * (kThreads * kVpt) + threadIdx.x) * V);
        __syncwarp();
      }
      if (lane == 0) {
        ws[parity][warp] = s;
        wt[parity][warp] = t;
      }
      __syncthreads();
      s = ws[parity][0];
      t = wt[parity][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        s += ws[parity][w];
        t += wt[parity][w];
      }
      parity ^= 1;
      const Stats part{m, s, t};
      if (splits == 1) {
        total = seg == 0 ? part : fold(total, part);
      } else if (threadIdx.x == 0) {
        seg_stats[seg - seg0] = part;
      }
      if constexpr (kTop) {
        int count = top.count;
        const bool full = count > kCandidates, end = seg + 1 == seg1;
        if (full) {
          top_overflow<T>(top, r, (static_cast<uint32_t>(seg) * (kThreads * kVpt) + threadIdx.x) * V, held, bound,
                          a.top);
          count = a.top;
        }
        if (full || end || count > kRankAbove) {
          rank_select(top.cand, count, a.top, top.list);
          __syncthreads();
          if (static_cast<int>(threadIdx.x) < a.top) top.cand[threadIdx.x] = top.list[threadIdx.x];
          count = end ? 0 : a.top;
          if (threadIdx.x == 0) top.count = count;
          // (not at the row's end, the list is full; an element of a later segment loses a tie)
          bound = max(bound, static_cast<uint32_t>(top.list[a.top - 1] >> 32) + 1);
          __syncthreads();
        }
        held = count;
      }
    }
    if (splits == 1) {
      write_row<T>(a, row, total, top.list);
      continue;
    }
    cluster_barrier();
    if (rank == 0) {
      const int ranks = (segments + per - 1) / per;     // that have a segment
      if constexpr (kTop) {
        if (threadIdx.x < kMaxTop) joined[threadIdx.x] = 0;
        for (int i = threadIdx.x; i < ranks * a.top; i += kThreads)
          top.cand[i] = remote_u64(remote(&top.list[i % a.top], i / a.top));
        __syncthreads();
        rank_select(top.cand, ranks * a.top, a.top, joined);
      }
      for (int seg = threadIdx.x; seg < segments; seg += kThreads) {
        const uint32_t at = remote(&seg_stats[seg % per], seg / per);
        all_stats[seg] = {remote_f32(at), remote_f32(at + 4), remote_f32(at + 8)};
      }
      __syncthreads();
      total = all_stats[0];
      for (int seg = 1; seg < segments; ++seg) total = fold(total, all_stats[seg]);
      write_row<T>(a, row, total, joined);
    }
    cluster_barrier();                                  // (read before it is written again)
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_backward_kernel(LogprobsGradArgs a) {
  constexpr int V = Elem<T>::kVec;
  constexpr int kUnroll = 4;
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * gridDim.y;
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  T* dx = static_cast<T*>(a.dlogits) + row * a.ldd;
  const int64_t vec0 = int64_t(blockIdx.x) * (kThreads * kUnroll) + threadIdx.x;
  uint4 r[kUnroll];
  load_vecs<T, kUnroll>(x, a.vocab, vec0, kThreads, Elem<T>::kNegInf, r);
  const float m = a.stats[2 * row], s = a.stats[2 * row + 1];
  const int64_t token = a.tokens[row];
  float g = a.dlogprobs ? a.dlogprobs[row] : 0.f;
  if (token < 0 || token >= a.vocab || s == 0.f) g = 0.f;   // no token, or no distribution
  const float h = a.dentropy && s != 0.f ? a.dentropy[row] : 0.f;
  const float ref = m == -INFINITY ? 0.f : m;
  const float inv = s == 0.f ? 0.f : 1.0f / s;
  // g + h (log p + entropy) = c + h (x - m)
  const float c = h != 0.f ? g + h * (a.entropy[row] - logf(s)) : g;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t vec = vec0 + i * kThreads;
    if ((vec & ~31ll) * V >= a.vocab) break;            // (uniform in the warp)
    float f[V];
    Elem<T>::unpack(r[i], f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = max_nan(f[e] - ref, kLowest);
      const float p = exp2_approx(d * kLog2e) * inv;
      f[e] = -p * fmaf(h, d, c);
    }
    const int64_t at = token - vec * V;
    if (at >= 0 && at < V) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e == at) f[e] += g;
    }
    store_vec(dx, a.vocab, vec, Elem<T>::pack(f));
  }
}

constexpr int64_t kResident = kBlocksPerSm * 152;                  // blocks that a GB300 holds at once
constexpr int64_t kSplitBelow = 2 * kResident;
constexpr int64_t kMaxGridY = 65535;                               // (y times z: more rows than there can be)

template <typename T, bool kTop, bool kPlain>
cudaError_t launch_forward(const LogprobsArgs& a, int segments, int per, int splits, cudaStream_t stream) {
  constexpr size_t kSmem = size_t(kStages) * kVpt * kThreads * 16;
  static PerDeviceOnce once;
  cudaError_t e = once.run([](int) {
    const auto kernel = logprobs_forward_kernel<T, kTop, kPlain>;
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    // (three blocks to an SM need all of its shared memory)
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    return r;
  });
  if (e != cudaSuccess) return e;
  const int64_t most = kResident / splits;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(static_cast<unsigned>((a.rows < most ? a.rows : most) * splits));
  config.blockDim = dim3(kThreads);
  config.dynamicSmemBytes = kSmem;
  config.stream = stream;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = static_cast<unsigned>(splits);
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  config.attrs = &cluster;
  config.numAttrs = splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&config, logprobs_forward_kernel<T, kTop, kPlain>, a, segments, per, splits);
  note_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t forward(const LogprobsArgs& a, cudaStream_t stream) {
  const int64_t seg_elems = segment_elems<T>();
  const int segments = static_cast<int>((a.vocab + seg_elems - 1) / seg_elems);
  // A cluster of 2, 4 or 8 blocks per row where the rows alone would leave
  // blocks without work (or badly spread over the last of few rounds).  Of 57
  // clusters of 8, the most, 51 are resident at once: bf16 131072 with 20
  // alternatives takes 13.2 us for 48 rows, 20.5 for 57 and for 64.
  int splits = 1;
  while (splits < kMaxSplits && splits < segments && a.rows * splits < kSplitBelow) splits *= 2;
  int per = (segments + splits - 1) / splits;
  if (per > kMaxPer) splits = 1, per = segments;        // (more than a block keeps for the others)
  if (plain_rows<T>(a.logits, a.ld, a.rows, a.vocab)) {
    if (a.top > 0) return launch_forward<T, true, true>(a, segments, per, splits, stream);
    return launch_forward<T, false, true>(a, segments, per, splits, stream);
  }
  if (a.top > 0) return launch_forward<T, true, false>(a, segments, per, splits, stream);
  return launch_forward<T, false, false>(a, segments, per, splits, stream);
}

template <typename T>
cudaError_t backward(const LogprobsGradArgs& a, cudaStream_t stream) {
  const int64_t span = int64_t(kThreads) * 4 * Elem<T>::kVec;
  const unsigned gy = static_cast<unsigned>(a.rows < kMaxGridY ? a.rows : kMaxGridY);
  const dim3 grid(static_cast<unsigned>((a.vocab + span - 1) / span), gy,
                  static_cast<unsigned>((a.rows + gy - 1) / gy));
  logprobs_backward_kernel<T><<<grid, kThreads, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs_forward(const LogprobsArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return a.bf16 ? forward<bf16>(a, stream) : forward<float>(a, stream);
}

cudaError_t launch_logprobs_backward(const LogprobsGradArgs& a, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return a.bf16 ? backward<bf16>(a, stream) : backward<float>(a, stream);
}

}  // namespace det
