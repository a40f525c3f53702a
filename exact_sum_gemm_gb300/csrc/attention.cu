// Attention, forward and backward, on the CUDA cores: f32 with short rows (the
// rest runs on the tensor cores, attention_tc.cu and attention_wide.cu), and
// the repair of what the tensor-core kernels leave.
//
//   s_ij = scale q_i . k_j over the visible pairs,  lse_i = log sum_j exp(s_ij)
//   p_ij = exp(s_ij - lse_i),  o_i = sum_j p_ij v_j
//   D_i = do_i . o_i,  dv_j = sum_i p_ij do_i,  ds_ij = p_ij (do_i . v_j - D_i) scale
//   dq_i = sum_j ds_ij k_j,  dk_j = sum_i ds_ij q_i
//
// Key j is visible to query i if j < k_lengths[batch] and, where causal,
// j <= i + lk - lq (the last query sees the last key).  A query that sees no
// key has output 0, lse -inf and no gradient.  Nothing that a mask hides
// reaches a result, NaN and infinities included: hidden keys past the length
// are read as zero, and a tile that the causal diagonal crosses and that holds
// a non-finite value is multiplied pair by visible pair.
//
// The probabilities are never stored: forward keeps a running maximum and sum
// per query, backward recomputes p from lse, at most 1: the rounding of lse and
// of s, of any size where scores are large, could make p infinite (the cap
// costs 0.4 % of 2 x 4096 causal, 16/4 heads of 128, 1.7 % with 16/16 of 64).  dk and dv are summed by the
// block that owns the keys, over the queries of all heads that share them, and
// dq by the block that owns the queries; s and do . v are computed twice for
// that, but no sum is taken by atomics, so results repeat bit for bit.  Each
// order of summation is a function of the lengths alone.
//
// 64 x 64 tiles, 256 threads as 16 x 16, f32 throughout.  In the products over
// the head dimension a thread has rows ty + 16 a and columns tx + 16 b and
// reads 4 values along the dimension at once: 8 shared 16-byte loads for 64
// multiply-adds, in rows padded by 16 bytes so that no two lanes' rows share
// banks.
//
// What bounds it at the sizes it is used at is latency: 33 rows of 4 heads of
// 64 are 4 blocks forward and 8 backward, 8.4 and 13.1 us, in calls that cost
// the host 17 and 26 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "det_train.h"
#include "rows.cuh"

namespace det {
namespace {

typedef __nv_bfloat16 bf16;

constexpr int kTile = 64;
constexpr int kThreads = 256;
constexpr int kPStride = kTile + 4;

// What a block needs to know of its (batch, head) pair.
struct Mask {
  int lq, keys, offset, causal;      // visible: i < lq, j < keys, !causal or j <= i + offset
  __device__ __forceinline__ bool sees(int i, int j) const {
    return i < lq && j < keys && (!causal || j <= i + offset);
  }
  // Whether the causal diagonal crosses the tile of queries i0 .. and keys j0 ..
  __device__ __forceinline__ bool crosses(int i0, int j0) const {
    return causal && j0 + kTile - 1 > i0 + offset;
  }
};

__device__ __forceinline__ Mask mask_of(const AttentionArgs& a, int batch) {
  Mask m;
  m.lq = a.lq;
  m.keys = a.lk;
  if (a.k_lengths) m.keys = max(0, min(a.lk, __ldg(a.k_lengths + batch)));
  m.offset = a.lk - a.lq;
  m.causal = a.causal;
  return m;
}

template <typename T>
__device__ __forceinline__ T* head_ptr(const Heads& h, int batch, int head) {
  return static_cast<T*>(h.p) + int64_t(batch) * h.sb + int64_t(head) * h.sh;
}

// (values that the split leaves out count as non-finite: a few next to FLT_MAX)
__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= kMostSplit; }

// Rows row0 .. row0 + 63 of one head to shared memory as f32, rows at or past
// `rows` and columns at or past `dim` as zero.  Whether any value is not finite.
template <typename T, int DP>
__device__ __forceinline__ bool load_tile(float* dst, const T* src, int64_t stride, int row0, int rows,
                                          int dim) {
  constexpr int kStride = DP + 4;
  constexpr uintptr_t kBytes = 4 * sizeof(T);
  const bool vec = dim % 4 == 0 &&
                   ((reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(stride * sizeof(T))) %
                    kBytes) == 0;
  bool bad = false;
#pragma unroll 4
  for (int c = threadIdx.x; c < kTile * DP / 4; c += kThreads) {
    const int r = c / (DP / 4), d = (c % (DP / 4)) * 4;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (row0 + r < rows) {
      const T* p = src + (row0 + r) * stride + d;
      if (vec && d < dim) {
        if constexpr (sizeof(T) == 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p));
          f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
          f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (d + e < dim) f[e] = Elem<T>::to_float(p[e]);
      }
    }
    bad |= !(finite(f[0]) && finite(f[1]) && finite(f[2]) && finite(f[3]));
    *reinterpret_cast<float4*>(dst + r * kStride + d) = make_float4(f[0], f[1], f[2], f[3]);
  }
  return bad;
}

// acc[a][b] = A(ty + 16 a) . B(tx + 16 b) over DP values.
template <int DP>
__device__ __forceinline__ void dot_rows(const float* A, const float* B, float (&acc)[4][4]) {
  constexpr int kStride = DP + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * kStride + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kStride + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
}

// acc[a][4 c + e] += sum_j P(ty + 16 a, j) B(j, 64 c + 4 tx + e).  kExact: only
// over the pairs that the mask shows (queries i0 .., keys j0 ..).
template <int DP, bool kExact>
__device__ __forceinline__ void rows_times(const float* P, const float* B, float (&acc)[4][DP / 16],
                                           const Mask& mask, int i0, int j0) {
  constexpr int kStride = DP + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int keys = min(kTile, mask.keys - j0);          // (P is 0 past them)
#pragma unroll 2
  for (int j = 0; j < keys; j += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * kPStride + j);
      p[i][0] = v.x, p[i][1] = v.y, p[i][2] = v.z, p[i][3] = v.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const float4 b = *reinterpret_cast<const float4*>(B + (j + jj) * kStride + 64 * c + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kExact && !mask.sees(i0 + ty + 16 * i, j0 + j + jj)) continue;
          acc[i][4 * c] = fmaf(p[i][jj], b.x, acc[i][4 * c]);
          acc[i][4 * c + 1] = fmaf(p[i][jj], b.y, acc[i][4 * c + 1]);
          acc[i][4 * c + 2] = fmaf(p[i][jj], b.z, acc[i][4 * c + 2]);
          acc[i][4 * c + 3] = fmaf(p[i][jj], b.w, acc[i][4 * c + 3]);
        }
      }
  }
}

// acc[a][4 c + e] += sum_i P(i, 4 ty + a) B(i, 64 c + 4 tx + e): P transposed.
template <int DP, bool kExact>
__device__ __forceinline__ void columns_times(const float* P, const float* B,
                                              float (&acc)[4][DP / 16], const Mask& mask, int i0,
                                              int j0) {
  constexpr int kStride = DP + 4;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int queries = min(kTile, mask.lq - i0);         // (P is 0 past them)
#pragma unroll 4
  for (int i = 0; i < queries; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(P + i * kPStride + 4 * ty);
    const float p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const float4 b = *reinterpret_cast<const float4*>(B + i * kStride + 64 * c + 4 * tx);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kExact && !mask.sees(i0 + i, j0 + 4 * ty + j)) continue;
        acc[j][4 * c] = fmaf(p[j], b.x, acc[j][4 * c]);
        acc[j][4 * c + 1] = fmaf(p[j], b.y, acc[j][4 * c + 1]);
        acc[j][4 * c + 2] = fmaf(p[j], b.z, acc[j][4 * c + 2]);
        acc[j][4 * c + 3] = fmaf(p[j], b.w, acc[j][4 * c + 3]);
      }
    }
  }
}

// Row `row` of a head: values acc[4 c + e] scaled to columns 64 c + 4 tx + e.
template <typename T, int DP>
__device__ __forceinline__ void store_row(T* dst, int64_t stride, int row, int dim,
                                          const float (&acc)[DP / 16], float by) {
  const int tx = threadIdx.x & 15;
  T* p = dst + row * stride;
#pragma unroll
  for (int c = 0; c < DP / 64; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 64 * c + 4 * tx + e;
      if (d < dim) p[d] = Elem<T>::from_float(acc[4 * c + e] * by);
    }
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The (tile, head, batch) of number `id`; tiles in descending order, so that
// the long rows of a causal mask start first.
__device__ __forceinline__ void place(int64_t id, int tiles, int heads, int& tile, int& head, int& batch) {
  const int64_t rest = id / (int64_t(heads));
  head = static_cast<int>(id - rest * heads);
  batch = static_cast<int>(rest / tiles);
  tile = tiles - 1 - static_cast<int>(rest - int64_t(batch) * tiles);
}

// Whether the tensor-core kernels flagged the tile that holds row `row`.
__device__ __forceinline__ bool flagged(const AttentionArgs& a, int rows, int heads, int row, int head,
                                        int batch) {
  if (a.flag_rows == 0) return true;
  const int tiles = (rows + a.flag_rows - 1) / a.flag_rows;
  return a.flags[(int64_t(batch) * tiles + row / a.flag_rows) * heads + head] != 0;
}

// Repair of a flagged tile: rows of `tile` (in shared memory) that hold a
// non-finite value, one bit each.  Called by the whole block.
template <int DP>
__device__ __forceinline__ uint64_t bad_rows(const float* tile, uint64_t* mask) {
  __syncthreads();
  if (threadIdx.x == 0) *mask = 0;
  __syncthreads();
  if (threadIdx.x < kTile) {
    bool bad = false;
    for (int d = 0; d < DP; ++d) bad |= !finite(tile[threadIdx.x * (DP + 4) + d]);
    if (bad) atomicOr(reinterpret_cast<unsigned long long*>(mask), 1ull << threadIdx.x);
  }
  __syncthreads();
  return *mask;
}

// kRepair: only rows that hold or see a non-finite value are written (flagged
// tiles).
template <typename T, int DP, bool kRepair>
__device__ __forceinline__ void forward_tile(const AttentionArgs& a, int64_t id) {
  constexpr int kStride = DP + 4;
  extern __shared__ float smem[];
  __shared__ uint64_t bad_mask;
  float* Q = smem;
  float* KV = Q + kTile * kStride;
  float* P = KV + kTile * kStride;
  int tile, h, b;
  place(id, (a.lq + kTile - 1) / kTile, a.hq, tile, h, b);
  const int hk = h / (a.hq / a.hkv), i0 = tile * kTile;
  if (kRepair && !flagged(a, a.lq, a.hq, i0, h, b)) return;
  bool affected[4] = {!kRepair, !kRepair, !kRepair, !kRepair};
  __syncthreads();
  const Mask mask = mask_of(a, b);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const T* k = head_ptr<const T>(a.k, b, hk);
  const T* v = head_ptr<const T>(a.v, b, hk);
  load_tile<T, DP>(Q, head_ptr<const T>(a.q, b, h), a.q.sl, i0, a.lq, a.dim);
  if (kRepair) {
    const uint64_t which = bad_rows<DP>(Q, &bad_mask);
#pragma unroll
    for (int i = 0; i < 4; ++i) affected[i] |= which >> (ty + 16 * i) & 1;
  }
  // rows that see a non-finite row of the key tile in KV
  auto mark = [&](int j0) {
    const uint64_t which = bad_rows<DP>(KV, &bad_mask);
    for (int j = 0; j < kTile; ++j)
      if (which >> j & 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) affected[i] |= mask.sees(i0 + ty + 16 * i, j0 + j);
  };
  const float c = a.scale * kLog2e;
  int end = mask.keys;
  if (mask.causal) end = max(0, min(end, min(i0 + kTile, a.lq) + mask.offset));
  float o[4][DP / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) o[i][d] = 0.f;
  }
  for (int j0 = 0; j0 < end; j0 += kTile) {
    __syncthreads();
    const bool bad_k = load_tile<T, DP>(KV, k, a.k.sl, j0, mask.keys, a.dim);
    if (kRepair) {
      if (__syncthreads_or(bad_k)) mark(j0);
    } else {
      __syncthreads();
    }
    float s[4][4];
    dot_rows<DP>(Q, KV, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = mask.sees(i0 + ty + 16 * i, j0 + tx + 16 * j) ? s[i][j] * c : -INFINITY;
        top = max_nan(top, s[i][j]);
      }
      top = max_nan(m[i], half_warp_max(top));
      const float ref = top == -INFINITY ? 0.f : top;
      const float by = exp2_approx(m[i] - ref);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2_approx(s[i][j] - ref);
        P[(ty + 16 * i) * kPStride + tx + 16 * j] = p;
        sum += p;
      }
      l[i] = l[i] * by + half_warp_sum(sum);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) o[i][d] *= by;
    }
    __syncthreads();
    const bool bad = __syncthreads_or(load_tile<T, DP>(KV, v, a.v.sl, j0, mask.keys, a.dim));
    if (kRepair && bad) mark(j0);
    if (bad && mask.crosses(i0, j0)) {
      rows_times<DP, true>(P, KV, o, mask, i0, j0);
    } else {
      rows_times<DP, false>(P, KV, o, mask, i0, j0);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i0 + ty + 16 * i;
    if (row < a.lq && affected[i]) {
      store_row<T, DP>(head_ptr<T>(a.o, b, h), a.o.sl, row, a.dim, o[i], l[i] == 0.f ? 0.f : 1.0f / l[i]);
      if (tx == 0)
        a.lse[(int64_t(b) * a.hq + h) * a.lq + row] =
            l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attention_forward_kernel(AttentionArgs a) {
  forward_tile<T, DP, false>(a, blockIdx.x);
}
// Whether any of `n` flags is set, asked by the whole block.
__device__ __forceinline__ bool any_flag(const int* flags, int64_t n) {
  bool any = false;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) any |= flags[i] != 0;
  return __syncthreads_or(any);
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attention_forward_repair_kernel(AttentionArgs a, int64_t flags,
                                                                            int64_t count) {
  if (!any_flag(a.flags, flags)) return;
  for (int64_t id = blockIdx.x; id < count; id += gridDim.x) forward_tile<T, DP, true>(a, id);
}

// x . y over dim elements, by one thread.
template <typename T>
__device__ __forceinline__ float row_dot(const T* x, const T* y, int dim) {
  float s = 0.f;
#pragma unroll 4
  for (int d = 0; d < dim; d += 8) {
    float f[8], g[8];
    load8(x, d, dim, f);
    load8(y, d, dim, g);
    s += dot8(f, g);
  }
  return s;
}

// A lane's share of delta = sum_j p_j do . v_j over the keys 0 .. few - 1 that
// are all the query sees: a key to a lane, its rows read whole by that thread.
// (8 elements a lane, as above, make a chain of loads and sums over the lanes
// that took twice as long.)  Not inlined: its registers would cost the other
// queries half of their blocks.
__device__ __noinline__ float delta_of_few(const AttentionArgs& a, int b, int h, int i, int few, float lse2) {
  const bf16* q = head_ptr<const bf16>(a.q, b, h) + i * a.q.sl;
  const bf16* g = head_ptr<const bf16>(a.dout, b, h) + i * a.dout.sl;
  const bf16* k = head_ptr<const bf16>(a.k, b, h / (a.hq / a.hkv));
  const bf16* v = head_ptr<const bf16>(a.v, b, h / (a.hq / a.hkv));
  float s = 0.f;
  for (int j = threadIdx.x & 15; j < few; j += 16) {
    const float p = probability(fmaf(row_dot(q, k + j * a.k.sl, a.dim), a.scale * kLog2e, -lse2));
    s = fmaf(p, row_dot(g, v + j * a.v.sl, a.dim), s);
  }
  return s;
}

// delta and lse2 of every query, bf16: 16 lanes per query, 8 elements each.
//
// delta is do . o (f32 takes it with the split of dO into planes).  bf16 has o
// only rounded, and where a query sees few keys
// that error is large beside do . v - delta, which is 0 for a single key: two
// keys' gradients are 3.4e-3 of their size off with it, and 1.7e-3 by the
// rounding of dS alone.  Such queries take delta from its other form.  At 16
// keys the two are 1.9e-3 and 1.7e-3, at 64 they are equal.  It costs 4 us of
// the 434 that the gradients of 2 x 4096 causal queries take (this kernel 25);
// up to 32 keys it would be 14.
constexpr int kFewKeys = 16;
__global__ void __launch_bounds__(kThreads, 6) attention_delta_kernel(__grid_constant__ const AttentionArgs a) {
  const int64_t id = int64_t(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4);
  const int d = (threadIdx.x & 15) * 8;
  // heads fastest: neighbouring lanes read neighbouring memory; then batches, so
  // that the queries of few keys of all of them come first and delay no end
  const int64_t rest = id / a.hq, row = rest / a.batch;
  const int h = static_cast<int>(id - rest * a.hq), b = static_cast<int>(rest - row * a.batch);
  const bool slot = row < a.stat_stride, valid = row < a.lq;
  const int i = static_cast<int>(row);
  float s = 0.f, lse2 = INFINITY;
  if (valid) {
    lse2 = __ldg(a.lse + (int64_t(b) * a.hq + h) * a.lq + i) * kLog2e;
    if (lse2 == -INFINITY) lse2 = INFINITY;
    float o[8], g[8];
    load8(head_ptr<const bf16>(a.o, b, h) + i * a.o.sl, d, a.dim, o);
    load8(head_ptr<const bf16>(a.dout, b, h) + i * a.dout.sl, d, a.dim, g);
    s = dot8(o, g);
    const Mask mask = mask_of(a, b);
    const int seen = mask.causal ? min(mask.keys, i + mask.offset + 1) : mask.keys;
    if (seen > 0 && seen <= kFewKeys) s = delta_of_few(a, b, h, i, seen, lse2);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (slot && (threadIdx.x & 15) == 0) {
    const int64_t at = (int64_t(b) * a.hq + h) * a.stat_stride + i;
    a.delta[at] = s;
    a.lse2[at] = lse2;
  }
}

// lse2 and delta of queries i0 .. i0 + 63, by 4 threads each, for the kernels
// below where they are the whole backward pass: at their few rows the launch
// above and its scratch would take longer than taking these again per tile.
template <typename T>
__device__ __forceinline__ void own_statistics(const AttentionArgs& a, int b, int h, int i0, float* lse2,
                                               float* delta) {
  static_assert(kThreads == 4 * kTile);
  const int r = threadIdx.x >> 2, i = i0 + r;
  float s = 0.f, top = INFINITY;
  if (i < a.lq) {
    top = __ldg(a.lse + (int64_t(b) * a.hq + h) * a.lq + i) * kLog2e;
    if (top == -INFINITY) top = INFINITY;
    const T* o = head_ptr<const T>(a.o, b, h) + i * a.o.sl;
    const T* g = head_ptr<const T>(a.dout, b, h) + i * a.dout.sl;
    for (int d = (threadIdx.x & 3) * 8; d < a.dim; d += 32) {
      float x[8], y[8];
      load8(o, d, a.dim, x);
      load8(g, d, a.dim, y);
      s += dot8(x, y);
    }
  }
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
  s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
  if ((threadIdx.x & 3) == 0) {
    lse2[r] = top;
    delta[r] = s;
  }
}

// p and ds of the thread's pairs from s and do . v.
__device__ __forceinline__ void probabilities(float (&s)[4][4], float (&dp)[4][4], const Mask& mask,
                                              int i0, int j0, const float* lse2, const float* delta,
                                              float c) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float top = lse2[ty + 16 * i], del = delta[ty + 16 * i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool seen = top != INFINITY && mask.sees(i0 + ty + 16 * i, j0 + tx + 16 * j);
      const float p = probability(fmaf(s[i][j], c, -top));
      s[i][j] = seen ? p : 0.f;
      dp[i][j] = seen ? p * (dp[i][j] - del) : 0.f;
    }
  }
}

__device__ __forceinline__ void put_pairs(float* P, const float (&v)[4][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) P[(ty + 16 * i) * kPStride + tx + 16 * j] = v[i][j];
}

template <typename T, int DP, bool kRepair>
__device__ __forceinline__ void dkv_tile(const AttentionArgs& a, int64_t id) {
  constexpr int kStride = DP + 4;
  extern __shared__ float smem[];
  __shared__ uint64_t bad_mask;
  float* K = smem;
  float* V = K + kTile * kStride;
  float* Q = V + kTile * kStride;
  float* G = Q + kTile * kStride;
  float* P = G + kTile * kStride;
  __shared__ float lse2[kTile], delta[kTile];
  int tile, hk, b;
  place(id, (a.lk + kTile - 1) / kTile, a.hkv, tile, hk, b);
  tile = (a.lk + kTile - 1) / kTile - 1 - tile;           // the first keys are seen most
  const int j0 = tile * kTile, share = a.hq / a.hkv;
  if (kRepair && !flagged(a, a.lk, a.hkv, j0, hk, b)) return;
  bool affected[4] = {!kRepair, !kRepair, !kRepair, !kRepair};
  __syncthreads();
  const Mask mask = mask_of(a, b);
  const int ty = threadIdx.x >> 4;
  float dk[4][DP / 16], dv[4][DP / 16];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) dk[j][d] = dv[j][d] = 0.f;
  if (j0 < mask.keys) {
    load_tile<T, DP>(K, head_ptr<const T>(a.k, b, hk), a.k.sl, j0, mask.keys, a.dim);
    load_tile<T, DP>(V, head_ptr<const T>(a.v, b, hk), a.v.sl, j0, mask.keys, a.dim);
    if (kRepair) {
      const uint64_t which = bad_rows<DP>(K, &bad_mask);
      const uint64_t both = which | bad_rows<DP>(V, &bad_mask);
#pragma unroll
      for (int j = 0; j < 4; ++j) affected[j] |= both >> (4 * ty + j) & 1;
    }
    const float c = a.scale * kLog2e;
    // the first tile of queries that sees any of these keys
    int first = 0;
    if (mask.causal) first = max(0, j0 - mask.offset) / kTile * kTile;
    for (int h = hk * share; h < (hk + 1) * share; ++h) {
      const T* q = head_ptr<const T>(a.q, b, h);
      const T* g = head_ptr<const T>(a.dout, b, h);
      const int64_t stats = (int64_t(b) * a.hq + h) * a.stat_stride;
      for (int i0 = first; i0 < a.lq; i0 += kTile) {
        __syncthreads();
        bool bad = load_tile<T, DP>(Q, q, a.q.sl, i0, a.lq, a.dim);
        bad |= load_tile<T, DP>(G, g, a.dout.sl, i0, a.lq, a.dim);
        if constexpr (!kRepair) {
          own_statistics<T>(a, b, h, i0, lse2, delta);
        } else if (threadIdx.x < kTile) {
          lse2[threadIdx.x] = a.lse2[stats + i0 + threadIdx.x];
          delta[threadIdx.x] = a.delta[stats + i0 + threadIdx.x];
        }
        bad = __syncthreads_or(bad);
        if (kRepair && bad) {
          const uint64_t which = bad_rows<DP>(Q, &bad_mask);
          const uint64_t both = which | bad_rows<DP>(G, &bad_mask);
          for (int i = 0; i < kTile; ++i)
            if (both >> i & 1)
#pragma unroll
              for (int j = 0; j < 4; ++j) affected[j] |= mask.sees(i0 + i, j0 + 4 * ty + j);
        }
        const bool exact = bad && mask.crosses(i0, j0);
        float s[4][4], dp[4][4];
        dot_rows<DP>(Q, K, s);
        dot_rows<DP>(G, V, dp);
        probabilities(s, dp, mask, i0, j0, lse2, delta, c);
        put_pairs(P, s);
        __syncthreads();
        if (exact) columns_times<DP, true>(P, G, dv, mask, i0, j0);
        else columns_times<DP, false>(P, G, dv, mask, i0, j0);
        __syncthreads();
        put_pairs(P, dp);
        __syncthreads();
        if (exact) columns_times<DP, true>(P, Q, dk, mask, i0, j0);
        else columns_times<DP, false>(P, Q, dk, mask, i0, j0);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = j0 + 4 * ty + j;
    if (row < a.lk && affected[j]) {
      if (row >= mask.keys) {                             // a hidden key: exactly zero
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) dk[j][d] = dv[j][d] = 0.f;
      }
      store_row<T, DP>(head_ptr<T>(a.dk, b, hk), a.dk.sl, row, a.dim, dk[j], a.scale);
      store_row<T, DP>(head_ptr<T>(a.dv, b, hk), a.dv.sl, row, a.dim, dv[j], 1.0f);
    }
  }
}

template <typename T, int DP, bool kRepair>
__device__ __forceinline__ void dq_tile(const AttentionArgs& a, int64_t id) {
  constexpr int kStride = DP + 4;
  extern __shared__ float smem[];
  __shared__ uint64_t bad_mask;
  float* Q = smem;
  float* G = Q + kTile * kStride;
  float* K = G + kTile * kStride;
  float* V = K + kTile * kStride;
  float* P = V + kTile * kStride;
  __shared__ float lse2[kTile], delta[kTile];
  int tile, h, b;
  place(id, (a.lq + kTile - 1) / kTile, a.hq, tile, h, b);
  const int hk = h / (a.hq / a.hkv), i0 = tile * kTile;
  if (kRepair && !flagged(a, a.lq, a.hq, i0, h, b)) return;
  bool affected[4] = {!kRepair, !kRepair, !kRepair, !kRepair};
  __syncthreads();
  const Mask mask = mask_of(a, b);
  const int ty = threadIdx.x >> 4;
  const T* k = head_ptr<const T>(a.k, b, hk);
  const T* v = head_ptr<const T>(a.v, b, hk);
  load_tile<T, DP>(Q, head_ptr<const T>(a.q, b, h), a.q.sl, i0, a.lq, a.dim);
  load_tile<T, DP>(G, head_ptr<const T>(a.dout, b, h), a.dout.sl, i0, a.lq, a.dim);
  if (kRepair) {
    const uint64_t which = bad_rows<DP>(Q, &bad_mask);
    const uint64_t both = which | bad_rows<DP>(G, &bad_mask);
#pragma unroll
    for (int i = 0; i < 4; ++i) affected[i] |= both >> (ty + 16 * i) & 1;
  }
  if constexpr (!kRepair) {
    own_statistics<T>(a, b, h, i0, lse2, delta);
  } else if (threadIdx.x < kTile) {
    const int64_t at = (int64_t(b) * a.hq + h) * a.stat_stride + i0 + threadIdx.x;
    lse2[threadIdx.x] = a.lse2[at];
    delta[threadIdx.x] = a.delta[at];
  }
  const float c = a.scale * kLog2e;
  int end = mask.keys;
  if (mask.causal) end = max(0, min(end, min(i0 + kTile, a.lq) + mask.offset));
  float dq[4][DP / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) dq[i][d] = 0.f;
  for (int j0 = 0; j0 < end; j0 += kTile) {
    __syncthreads();
    bool bad = load_tile<T, DP>(K, k, a.k.sl, j0, mask.keys, a.dim);
    bad |= load_tile<T, DP>(V, v, a.v.sl, j0, mask.keys, a.dim);
    bad = __syncthreads_or(bad);
    if (kRepair && bad) {
      const uint64_t which = bad_rows<DP>(K, &bad_mask);
      const uint64_t both = which | bad_rows<DP>(V, &bad_mask);
      for (int j = 0; j < kTile; ++j)
        if (both >> j & 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) affected[i] |= mask.sees(i0 + ty + 16 * i, j0 + j);
    }
    const bool exact = bad && mask.crosses(i0, j0);
    float s[4][4], dp[4][4];
    dot_rows<DP>(Q, K, s);
    dot_rows<DP>(G, V, dp);
    probabilities(s, dp, mask, i0, j0, lse2, delta, c);
    put_pairs(P, dp);
    __syncthreads();
    if (exact) rows_times<DP, true>(P, K, dq, mask, i0, j0);
    else rows_times<DP, false>(P, K, dq, mask, i0, j0);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i0 + ty + 16 * i;
    if (row < a.lq && affected[i])
      store_row<T, DP>(head_ptr<T>(a.dq, b, h), a.dq.sl, row, a.dim, dq[i], a.scale);
  }
}

// The key tiles and the query tiles in one launch (one after the other, two
// launches of few blocks took 34 us for 33 rows).
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attention_backward_kernel(AttentionArgs a, int64_t dkv_count) {
  if (blockIdx.x < dkv_count) dkv_tile<T, DP, false>(a, blockIdx.x);
  else dq_tile<T, DP, false>(a, blockIdx.x - dkv_count);
}
// The key tiles' flags first, then the query tiles'.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
    attention_backward_repair_kernel(AttentionArgs a, int64_t dkv_flags, int64_t dkv_count,
                                     int64_t dq_flags, int64_t dq_count) {
  if (!any_flag(a.flags, dkv_flags + dq_flags)) return;
  for (int64_t id = blockIdx.x; id < dkv_count; id += gridDim.x) dkv_tile<T, DP, true>(a, id);
  if (a.flag_rows != 0) a.flags += dkv_flags;
  for (int64_t id = blockIdx.x; id < dq_count; id += gridDim.x) dq_tile<T, DP, true>(a, id);
}

template <int DP>
constexpr int smem_bytes(int tiles) { return (tiles * kTile * (DP + 4) + kTile * kPStride) * 4; }

template <typename K, typename... Args>
cudaError_t launch(PerDeviceOnce& once, K kernel, int64_t blocks, int smem, cudaStream_t stream, Args... args) {
  cudaError_t e = once.run([&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(args...);
  note_launch();
  return cudaGetLastError();
}

int64_t tiles_of(int n) { return (int64_t(n) + kTile - 1) / kTile; }
int64_t tc_tiles(int n, int rows) { return (int64_t(n) + rows - 1) / rows; }

// Blocks of a repair launch: a few, as they rarely have anything to do; each
// looks at all flags first.
int64_t repair_blocks(int64_t count) { return count < 152 ? count : 152; }

// bf16 runs on the tensor cores at every size; the CUDA-core kernels then only
// repair the tiles that were flagged, which takes a causal mask.
template <int DP>
cudaError_t forward_bf16(const AttentionArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_attention_tc_forward(a, stream);
  if (e != cudaSuccess || !a.causal) return e;
  static PerDeviceOnce once;
  const int64_t count = tiles_of(a.lq) * a.hq * a.batch;
  return launch(once, attention_forward_repair_kernel<bf16, DP>, repair_blocks(count), smem_bytes<DP>(2),
                stream, a, tc_tiles(a.lq, a.flag_rows) * a.hq * a.batch, count);
}

// f32 on the tensor cores pays for its split and its three planes from about 64
// rows on: forward + backward, causal, on the tensor cores and on the CUDA
// cores, in us: 4 heads of 64, 64 rows: 24 and 26, 128 rows: 31 and 44, 512
// rows: 57 and 149; 4 x 16 heads of 64, 64 rows: 28 and 27, 512 rows: 128 and
// 394; 4 x 16 heads of 128, 64 rows: 37 and 42, 512 rows: 353 and 878.
constexpr int kSplitRows = 64;
bool split_pays(const AttentionArgs& a) {
  return !a.bf16 && a.lk >= kSplitRows && a.lq >= kSplitRows;
}
int64_t plane_bytes(const AttentionArgs& a, int64_t rows) {
  return 3 * rows * (a.dim > 64 ? 128 : 64) * int64_t(sizeof(bf16));
}

template <int DP>
cudaError_t forward_f32(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once;
  return launch(once, attention_forward_kernel<float, DP>, tiles_of(a.lq) * a.hq * a.batch,
                smem_bytes<DP>(2), stream, a);
}

// Scratch of the split: planes of `tensors` tensors and the flags; sets them.
size_t split_bytes(const AttentionArgs& a, int tensors) {
  const int64_t q = int64_t(a.batch) * a.hq * a.lq, k = int64_t(a.batch) * a.hkv * a.lk;
  return plane_bytes(a, q) * (tensors - 2) + plane_bytes(a, k) * 2 + attention_split_blocks(a) * tensors * sizeof(int);
}
void split_scratch(AttentionArgs& a, int tensors, char* p) {
  const int64_t q = int64_t(a.batch) * a.hq * a.lq, k = int64_t(a.batch) * a.hkv * a.lk;
  for (int t = 0; t < tensors; ++t) {
    a.planes[t] = p;
    p += plane_bytes(a, t == 1 || t == 2 ? k : q);
  }
  a.flags = reinterpret_cast<int*>(p);
  a.flag_rows = 0;
}

template <int DP>
cudaError_t forward_split(AttentionArgs a, cudaStream_t stream) {
  static PerDeviceOnce once;
  void* scratch = nullptr;
  cudaError_t e = pool_alloc(&scratch, split_bytes(a, 3), stream);
  if (e != cudaSuccess) return e;
  split_scratch(a, 3, static_cast<char*>(scratch));
  e = launch_attention_split(a, 3, stream);
  if (e == cudaSuccess) e = launch_attention_tc_forward(a, stream);
  const int64_t count = tiles_of(a.lq) * a.hq * a.batch;
  if (e == cudaSuccess)
    e = launch(once, attention_forward_repair_kernel<float, DP>, repair_blocks(count), smem_bytes<DP>(2), stream, a,
               attention_split_blocks(a) * 3, count);
  const cudaError_t f = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : f;
}

template <int DP>
cudaError_t backward_split(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = launch_attention_split(a, 4, stream);
  if (e == cudaSuccess) e = launch_attention_tc_backward(a, stream);
  const int64_t dkv_count = a.dk.p ? tiles_of(a.lk) * a.hkv * a.batch : 0;
  const int64_t dq_count = a.dq.p ? tiles_of(a.lq) * a.hq * a.batch : 0;
  if (e == cudaSuccess)
    e = launch(once, attention_backward_repair_kernel<float, DP>,
               repair_blocks(dkv_count > dq_count ? dkv_count : dq_count), smem_bytes<DP>(4), stream, a,
               attention_split_blocks(a) * 4, dkv_count, int64_t(0), dq_count);
  return e;
}

template <int DP>
cudaError_t backward_bf16(AttentionArgs a, int* flags, cudaStream_t stream) {
  static PerDeviceOnce once;
  const bool dkv = a.dk.p && a.lk > 0, dq = a.dq.p && a.lq > 0;
  const int64_t dkv_flags = dkv ? tc_tiles(a.lk, kTcBackwardRows) * a.hkv * a.batch : 0;
  const int64_t dq_flags = dq ? tc_tiles(a.lq, kTcBackwardRows) * a.hq * a.batch : 0;
  a.flag_rows = kTcBackwardRows;
  a.flags = flags;
  a.dq_flags = dkv_flags;
  cudaError_t e = launch_attention_tc_backward(a, stream);
  if (!flags || dkv_flags + dq_flags == 0 || e != cudaSuccess) return e;
  const int64_t dkv_count = dkv ? tiles_of(a.lk) * a.hkv * a.batch : 0;
  const int64_t dq_count = dq ? tiles_of(a.lq) * a.hq * a.batch : 0;
  return launch(once, attention_backward_repair_kernel<bf16, DP>,
                repair_blocks(dkv_count > dq_count ? dkv_count : dq_count), smem_bytes<DP>(4), stream, a,
                dkv_flags, dkv_count, dq_flags, dq_count);
}

template <int DP>
cudaError_t backward_f32(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once;
  const int64_t dkv = a.dk.p ? tiles_of(a.lk) * a.hkv * a.batch : 0;
  const int64_t dq = a.dq.p ? tiles_of(a.lq) * a.hq * a.batch : 0;
  if (dkv + dq == 0) return cudaSuccess;
  return launch(once, attention_backward_kernel<float, DP>, dkv + dq, smem_bytes<DP>(4), stream, a, dkv);
}

}  // namespace

cudaError_t launch_attention_forward(const AttentionArgs& args, cudaStream_t stream) {
  if (args.batch == 0 || args.lq == 0) return cudaSuccess;
  AttentionArgs a = args;
  a.halves = attention_halves(a);
  if (split_pays(a)) return a.dim <= 64 ? forward_split<64>(a, stream) : forward_split<128>(a, stream);
  if (!a.bf16) return a.dim <= 64 ? forward_f32<64>(a, stream) : forward_f32<128>(a, stream);
  void* scratch = nullptr;
  if (a.causal) {
    a.flag_rows = 128 * a.halves;
    const int64_t flags = tc_tiles(a.lq, a.flag_rows) * a.hq * a.batch;
    const cudaError_t e = pool_alloc(&scratch, size_t(flags) * sizeof(int), stream);
    if (e != cudaSuccess) return e;
    a.flags = static_cast<int*>(scratch);
  }
  const cudaError_t e = a.dim <= 64 ? forward_bf16<64>(a, stream) : forward_bf16<128>(a, stream);
  const cudaError_t f = scratch ? cudaFreeAsync(scratch, stream) : cudaSuccess;
  return e != cudaSuccess ? e : f;
}

cudaError_t launch_attention_backward(const AttentionArgs& args, cudaStream_t stream) {
  if (args.batch == 0 || (!args.dq.p && !args.dk.p)) return cudaSuccess;
  AttentionArgs a = args;
  if (!a.bf16 && !split_pays(a)) return a.dim <= 64 ? backward_f32<64>(a, stream) : backward_f32<128>(a, stream);
  a.stat_stride = (int64_t(a.lq) + 127) / 128 * 128;        // (whole tiles of every kernel)
  const int64_t rows = a.batch * a.hq * a.stat_stride;
  const size_t stat_bytes = (rows > 0 ? rows : 128) * sizeof(float);
  const int64_t flags = a.bf16 && a.causal ? (tc_tiles(a.lk, kTcBackwardRows) * a.hkv +
                                              tc_tiles(a.lq, kTcBackwardRows) * a.hq) * a.batch : 0;
  const size_t more = split_pays(a) ? split_bytes(a, 4) : size_t(flags) * sizeof(int);
  void* scratch = nullptr;
  cudaError_t e = pool_alloc(&scratch, 2 * stat_bytes + more, stream);
  if (e != cudaSuccess) return e;
  a.delta = static_cast<float*>(scratch);
  a.lse2 = reinterpret_cast<float*>(static_cast<char*>(scratch) + stat_bytes);
  int* flag_words = flags > 0 ? reinterpret_cast<int*>(static_cast<char*>(scratch) + 2 * stat_bytes) : nullptr;
  if (rows > 0 && a.bf16) {
    const unsigned grid = static_cast<unsigned>((rows + kThreads / 16 - 1) / (kThreads / 16));
    attention_delta_kernel<<<grid, kThreads, 0, stream>>>(a);
    note_launch();
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    if (a.bf16) e = a.dim <= 64 ? backward_bf16<64>(a, flag_words, stream) : backward_bf16<128>(a, flag_words, stream);
    else {
      split_scratch(a, 4, static_cast<char*>(scratch) + 2 * stat_bytes);
      e = a.dim <= 64 ? backward_split<64>(a, stream) : backward_split<128>(a, stream);
    }
  }
  const cudaError_t f = cudaFreeAsync(scratch, stream);
  return e != cudaSuccess ? e : f;
}

}  // namespace det
