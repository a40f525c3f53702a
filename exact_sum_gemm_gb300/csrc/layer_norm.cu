// Layer norm over the last axis, forward and backward.
//
//   mean = sum_c x / W,  rstd = 1 / sqrt(sum_c (x - mean)^2 / W + eps),
//   xhat = (x - mean) rstd,  y = xhat w + b
//   g = dy w,  dx = rstd (g - sum_c(g) / W - xhat sum_c(g xhat) / W)
//   dw = sum_rows dy xhat,  db = sum_rows dy
//
// All sums are f32.  Every order of summation is a function of (rows, W, type)
// alone: a row is owned by a warp or a block chosen by W, and the rows' sums
// for dw and db are taken by a fixed number of row groups and then over the
// groups in order.  So results repeat bit for bit, and y, dx and the
// statistics of a row do not depend on the other rows.
//
// The operator is bound by memory: forward reads x and writes y, backward
// reads dy and x and writes dx, each once, the row being kept in registers
// between its statistics and its result (32 bytes of it to a thread for bf16, 64
// for f32, in up to 4096 columns; twice that in more, where fewer threads make
// the sums over a block cheaper).  Rows on their way wait in shared memory, two
// ahead.  Measured, of the copy bandwidth of 6.69 TB/s: f32 16384 x 4096 forward
// 79 us (6.8 TB/s), backward 115 + 6 us (7.0 TB/s; the 6 are the reduction of
// dw and db over the blocks); bf16 8192 x 4096 27 us (5.0 TB/s) and 42 + 6 us
// (4.8 TB/s).  bf16 has half the time for the same instructions: forward they
// take 71 % of the issue slots, a block's two barriers a row being part of the
// rest.  Backward is bound by latency: 16 warps of 128 registers to an SM (22 %),
// 57 % of the issue slots, one barrier a row.  So are rows that do not start on
// 16 bytes (bf16 1111 x 5001 forward 17 us: 51 % of the slots, 8 % of DRAM): their
// vectors are loaded to registers, shifted into place and stored to the ring, so
// that a row to come is waited for before the present one is summed.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "det_train.h"
#include "rows.cuh"

namespace det {
namespace {

typedef __nv_bfloat16 bf16;

// V f32 values of vector `vec` (V elements) of a row of TW elements.
template <typename TW, int V>
__device__ __forceinline__ void load_f32(const TW* p, int64_t n, int64_t vec, float (&f)[V]) {
  if constexpr (Elem<TW>::kVec == V) {
    uint4 r[1];
    load_vecs<TW, 1>(p, n, vec, 0, 0u, r);
    Elem<TW>::unpack(r[0], f);
  } else {
    uint4 r[2];
    float a[4], b[4];
    load_vecs<TW, 2>(p, n, 2 * vec, 1, 0u, r);
    Elem<TW>::unpack(r[0], a);
    Elem<TW>::unpack(r[1], b);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  }
}
template <typename T>
__device__ __forceinline__ uint4 load_one(const T* p, int64_t n, int64_t vec) {
  uint4 r[1];
  load_vecs<T, 1>(p, n, vec, 0, 0u, r);
  return r[0];
}

// The thread's vectors of a parameter: kept in registers where it has the type
// of the rows, else read again (from L1) for every row.
template <typename TW, int V, int kVpt>
struct Parameter {
  static constexpr bool kKept = Elem<TW>::kVec == V;
  const TW* p;
  int64_t n;
  uint4 r[kKept ? kVpt : 1];
  __device__ __forceinline__ Parameter(const void* ptr, int64_t width, int lane, int stride)
      : p(static_cast<const TW*>(ptr)), n(width) {
    if constexpr (kKept) {
      if (p) load_vecs<TW, kVpt>(p, n, lane, stride, 0u, r);
    }
  }
  __device__ __forceinline__ void get(int i, int64_t vec, float (&f)[V]) const {
    if constexpr (kKept) Elem<TW>::unpack(r[i], f);
    else load_f32<TW, V>(p, n, vec, f);
  }
};

template <typename T, bool kPlain>
__device__ __forceinline__ void put_vec(T* p, int W, int vec, const uint4& v) {
  if constexpr (kPlain) {
    if (vec * Elem<T>::kVec < W) reinterpret_cast<uint4*>(p)[vec] = v;
  } else {
    store_vec(p, W, vec, v);
  }
}

constexpr int kElems = 16;                              // of a row per thread (forward: see there)
constexpr int kStages = 3;                              // rows on their way or in use

// Sum of the warps' values buf[0 .. kWarps - 1], in a fixed order.  16 warps and
// more read one each and add over the lanes: 32 reads and additions in every
// thread were a quarter of the instructions of a row.
template <int kWarps>
__device__ __forceinline__ float warps_sum(const float* buf) {
  if constexpr (kWarps >= 16) {
    const int lane = threadIdx.x & 31;
    return warp_sum(kWarps == 32 || lane < kWarps ? buf[lane] : 0.f);
  } else {
    float s = buf[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += buf[w];
    return s;
  }
}

// Sum over the kTpr threads that share a row, in a fixed order; every thread
// gets it.  kTpr = 32: the warp.  Otherwise the whole block, through `buf`
// (one float per warp); the caller alternates two buffers, so one barrier
// per sum is enough.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float* buf) {
  v = warp_sum(v);
  if constexpr (kTpr > 32) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warps_sum<kTpr / 32>(buf);
  }
  return v;
}

// Blocks to an SM: 768 threads of 16 elements, 512 of 32.
constexpr int forward_blocks(int threads, int elems) { return (elems == 16 ? 768 : 512) / threads; }

// kThreads / kTpr rows at a time per block, kElems elements of a row per thread;
// the rows to come are on their way in kStages - 1 stages of the ring.
// kPlain: rows of whole, aligned vectors (the general form costs about twice
// the instructions).  Both assign threads the same elements.
template <typename T, typename TW, int kThreads, int kTpr, int kElems, bool kPlain>
__global__ void __launch_bounds__(kThreads, forward_blocks(kThreads, kElems))
    layer_norm_forward_kernel(LayerNormArgs a) {
  constexpr int V = Elem<T>::kVec, kVpt = kElems / V;
  constexpr int kRows = kThreads / kTpr;
  extern __shared__ uint4 ring[];
  __shared__ float buf[2][32];
  const int lane = threadIdx.x % kTpr;
  const int W = static_cast<int>(a.width);
  const int64_t step = int64_t(gridDim.x) * kRows;
  const float inv_w = 1.0f / static_cast<float>(W);
  int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kTpr;
  uint4* slots = ring + threadIdx.x;
  auto fetch = [&](int64_t r, int stage) {
    if (r < a.rows)
      ring_load<T, kVpt, kPlain>(slots + stage * (kVpt * kThreads), kThreads,
                                 static_cast<const T*>(a.x) + r * a.ldx, W, lane, kTpr, 0u);
    ring_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(row + s * step, s);
  const Parameter<TW, V, kVpt> weight(a.weight, W, lane, kTpr), bias(a.bias, W, lane, kTpr);
  for (int stage = 0; row < a.rows; row += step) {
    fetch(row + (kStages - 1) * step, (stage + kStages - 1) % kStages);
    ring_wait<kStages - 1>();
    const uint4* v = slots + stage * (kVpt * kThreads);
    float f[kVpt][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      uint4 r = v[i * kThreads];
      if (kPlain && (lane + i * kTpr) * V >= W) r = make_uint4(0, 0, 0, 0);
      Elem<T>::unpack(r, f[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) s += f[i][e];
    }
    const float mean = row_sum<kTpr>(s, buf[0]) * inv_w;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      const int left = W - (lane + i * kTpr) * V;       // elements of the vector within the row
      if (kPlain) {
        if (left > 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f[i][e] -= mean;
            s += f[i][e] * f[i][e];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[i][e] = e < left ? f[i][e] - mean : 0.f;
          s += f[i][e] * f[i][e];
        }
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<kTpr>(s, buf[1]) * inv_w + a.eps);
    if (lane == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      const int vec = lane + i * kTpr;
      if ((vec & ~31) * V >= W) break;                  // (uniform in the warp)
      float w[V], b[V];
      if (a.weight) weight.get(i, vec, w);
      if (a.bias) bias.get(i, vec, b);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t = f[i][e] * rstd;
        if (a.weight) t *= w[e];
        if (a.bias) t += b[e];
        f[i][e] = t;
      }
      put_vec<T, kPlain>(y, W, vec, Elem<T>::pack(f[i]));
    }
    stage = (stage + 1) % kStages;
  }
}

// Rows too wide for registers: the row is read three times, from L2 after the
// first.
template <typename T, typename TW, int kThreads>
__global__ void __launch_bounds__(kThreads) layer_norm_forward_wide_kernel(LayerNormArgs a) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float buf[2][32];
  const int64_t row = blockIdx.x, W = a.width;
  const int64_t nvec = (W + V - 1) / V, nvec_warp = (nvec + 31) / 32 * 32;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  float v[V];
  float s = 0.f;
  for (int64_t vec = threadIdx.x; vec < nvec; vec += kThreads) {
    Elem<T>::unpack(load_one(x, W, vec), v);
#pragma unroll
    for (int e = 0; e < V; ++e) s += v[e];
  }
  const float mean = row_sum<kThreads>(s, buf[0]) / static_cast<float>(W);
  s = 0.f;
  for (int64_t vec = threadIdx.x; vec < nvec; vec += kThreads) {
    Elem<T>::unpack(load_one(x, W, vec), v);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = v[e] - mean;
      if (vec * V + e < W) s += d * d;
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<kThreads>(s, buf[1]) / static_cast<float>(W) + a.eps);
  if (threadIdx.x == 0) {
    a.mean[row] = mean;
    a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  for (int64_t vec = threadIdx.x; vec < nvec_warp; vec += kThreads) {
    float w[V], b[V];
    Elem<T>::unpack(load_one(x, W, vec), v);
    if (a.weight) load_f32<TW, V>(static_cast<const TW*>(a.weight), W, vec, w);
    if (a.bias) load_f32<TW, V>(static_cast<const TW*>(a.bias), W, vec, b);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float t = (v[e] - mean) * rstd;
      if (a.weight) t *= w[e];
      if (a.bias) t += b[e];
      v[e] = t;
    }
    store_vec(y, W, vec, Elem<T>::pack(v));
  }
}

// Rows that kTpr threads share backward are wider than this (see the dispatch).
constexpr int narrowest(int tpr) { return tpr == 32 ? 0 : tpr == 128 ? 512 : 8 * tpr; }

// Block `block` of `blocks` takes rows block, block + blocks, ... (times
// kThreads / kTpr rows at once), writes their dx and, with kSums, keeps its own
// sums of dy xhat and dy, written at the end as one row of the partial sums
// [blocks][2][W].  A thread owns the same columns in every row, so the sums
// stay in its registers; x and dy come through the ring.
template <typename T, typename TW, int kThreads, int kTpr, int kDepth, bool kSums, bool kPlain>
__device__ __forceinline__ void backward_rows(const LayerNormGradArgs& a, int block, int blocks) {
  constexpr int V = Elem<T>::kVec, kVpt = kElems / V;
  constexpr int kRows = kThreads / kTpr;
  constexpr int kWhole = narrowest(kTpr) / (kTpr * V);  // a thread's first vectors, never past the row's end
  // 1024 threads have 64 registers each: no room for a row beside the sums, so
  // that it is read from the ring again (16384 columns: 175 us with spills)
  constexpr bool kAgain = kThreads == 1024;
  extern __shared__ uint4 ring[];
  __shared__ float buf[2][2][32];
  const int lane = threadIdx.x % kTpr;
  const int W = static_cast<int>(a.width);
  const int64_t step = int64_t(blocks) * kRows;
  const float inv_w = 1.0f / static_cast<float>(W);
  float acc[kSums ? 2 * kVpt : 1][V];
#pragma unroll
  for (int i = 0; i < (kSums ? 2 * kVpt : 1); ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;

  int64_t row = int64_t(block) * kRows + threadIdx.x / kTpr;
  uint4* slots = ring + threadIdx.x;
  constexpr int kStage = 2 * kVpt * kThreads;
  float next_m = 0.f, next_rs = 0.f;                    // the next row's statistics
  auto fetch = [&](int64_t r, int stage) {
    if (r < a.rows) {
      uint4* to = slots + stage * kStage;
      ring_load<T, kVpt, kPlain>(to, kThreads, static_cast<const T*>(a.x) + r * a.ldx, W, lane, kTpr, 0u);
      ring_load<T, kVpt, kPlain>(to + kVpt * kThreads, kThreads, static_cast<const T*>(a.dy) + r * a.lddy, W,
                                 lane, kTpr, 0u);
    }
    ring_commit();
  };
  auto statistics = [&](int64_t r) {
    if (r < a.rows) {
      next_m = __ldg(a.mean + r);
      next_rs = __ldg(a.rstd + r);
    }
  };
#pragma unroll
  for (int s = 0; s < kDepth - 1; ++s) fetch(row + s * step, s);
  statistics(row);
  const Parameter<TW, V, kVpt> weight(a.weight, W, lane, kTpr);
  int parity = 0;
  for (int stage = 0; row < a.rows; row += step, parity ^= 1) {
    const float m = next_m, rs = next_rs;
    fetch(row + (kDepth - 1) * step, (stage + kDepth - 1) % kDepth);
    statistics(row + step);
    ring_wait<kDepth - 1>();
    const uint4* v = slots + stage * kStage;
    stage = (stage + 1) % kDepth;
    float s1 = 0.f, s2 = 0.f;
    // xhat and g = dy w of vector i
    auto read = [&](int i, float (&xh)[V], float (&dy)[V], float (&g)[V]) {
      // columns past the row's end have dy = 0 and xhat = 0 ((0 - m) rs may be infinite)
      const int left = W - (lane + i * kTpr) * V;       // elements of the vector within the row
      const bool past = kPlain && i >= kWhole && left <= 0;
      uint4 rx = v[i * kThreads], rd = v[(kVpt + i) * kThreads];
      if (past) rx = rd = make_uint4(0, 0, 0, 0);
      const float mean = past ? 0.f : m;
      Elem<T>::unpack(rx, xh);
      Elem<T>::unpack(rd, dy);
      float w[V];
      if (a.weight) weight.get(i, lane + i * kTpr, w);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[e] = (xh[e] - mean) * rs;
        g[e] = a.weight ? dy[e] * w[e] : dy[e];
      }
      if (!kPlain && i >= kWhole && left < V) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e >= left) xh[e] = 0.f;
      }
    };
    float xh[kVpt][V], g[kVpt][V];
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      float dy[V];
      read(i, xh[i], dy, g[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (kSums) {
          acc[kSums ? i : 0][e] += dy[e] * xh[i][e];
          acc[kSums ? kVpt + i : 0][e] += dy[e];
        }
        s1 += g[i][e];
        s2 += g[i][e] * xh[i][e];
      }
    }
    if (a.dx) {
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      if constexpr (kTpr > 32) {
        // (two buffers in turn: one barrier per row)
        if ((threadIdx.x & 31) == 0) {
          buf[parity][0][threadIdx.x >> 5] = s1;
          buf[parity][1][threadIdx.x >> 5] = s2;
        }
        __syncthreads();
        s1 = warps_sum<kTpr / 32>(buf[parity][0]);
        s2 = warps_sum<kTpr / 32>(buf[parity][1]);
      }
      const float c1 = s1 * inv_w, c2 = s2 * inv_w;
      T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
      for (int i = 0; i < kVpt; ++i) {
        const int vec = lane + i * kTpr;
        if ((vec & ~31) * V >= W) break;                // (uniform in the warp)
        float dy[V];
        if (kAgain) read(i, xh[i], dy, g[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) g[i][e] = rs * (g[i][e] - c1 - xh[i][e] * c2);
        put_vec<T, kPlain>(dx, W, vec, Elem<T>::pack(g[i]));
      }
    }
  }
  if constexpr (kSums) {
    float* part = a.partial + int64_t(block) * 2 * W;
    if constexpr (kTpr > 32) {
#pragma unroll
      for (int i = 0; i < kVpt; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = (lane + i * kTpr) * V + e;
          if (c < W) {
            part[c] = acc[i][e];
            part[W + c] = acc[kVpt + i][e];
          }
        }
    } else {
      // a warp per row: the block's warps are added in order
      float* sums = reinterpret_cast<float*>(ring);
      ring_wait<0>();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVpt; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e)
            sums[(threadIdx.x / 32) * (kVpt * V * 32) + (lane + i * 32) * V + e] = acc[h * kVpt + i][e];
        __syncthreads();
        for (int c = threadIdx.x; c < W; c += kThreads) {
          float t = sums[c];
#pragma unroll
          for (int w = 1; w < kRows; ++w) t += sums[w * (kVpt * V * 32) + c];
          part[h * W + c] = t;
        }
      }
    }
  }
}

template <typename T, typename TW, int kThreads, int kTpr, int kDepth, bool kPlain>
__global__ void __launch_bounds__(kThreads, kThreads >= 512 ? 1 : 512 / kThreads)
    layer_norm_backward_kernel(LayerNormGradArgs a) {
  backward_rows<T, TW, kThreads, kTpr, kDepth, true, kPlain>(a, blockIdx.x, gridDim.x);
}

// Few rows: one launch and no scratch.  The first `row_blocks` blocks write dx;
// each of the others owns kThreads columns and takes their sums over all rows.
template <typename T, typename TW, int kThreads, int kTpr>
__global__ void __launch_bounds__(kThreads) layer_norm_backward_few_kernel(LayerNormGradArgs a, int row_blocks) {
  if (static_cast<int>(blockIdx.x) < row_blocks) {
    backward_rows<T, TW, kThreads, kTpr, 1, false, false>(a, blockIdx.x, row_blocks);
    return;
  }
  const int64_t c = int64_t(blockIdx.x - row_blocks) * kThreads + threadIdx.x;
  if (c >= a.width) return;
  float sw = 0.f, sb = 0.f;
#pragma unroll 8
  for (int r = 0; r < static_cast<int>(a.rows); ++r) {
    const float dy = Elem<T>::to_float(static_cast<const T*>(a.dy)[r * a.lddy + c]);
    const float x = Elem<T>::to_float(static_cast<const T*>(a.x)[r * a.ldx + c]);
    sw += dy * ((x - __ldg(a.mean + r)) * __ldg(a.rstd + r));
    sb += dy;
  }
  if (a.dweight) static_cast<TW*>(a.dweight)[c] = Elem<TW>::from_float(sw);
  if (a.dbias) static_cast<TW*>(a.dbias)[c] = Elem<TW>::from_float(sb);
}

// Rows too wide for the kernel above: dx reads its row twice, and the sums
// over rows are taken by a kernel of their own (a thread per vector of
// columns, a fixed set of rows per block row).
template <typename T, typename TW, int kThreads>
__global__ void __launch_bounds__(kThreads) layer_norm_dx_wide_kernel(LayerNormGradArgs a) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float buf[2][32];
  const int64_t row = blockIdx.x, W = a.width;
  const int64_t nvec = (W + V - 1) / V, nvec_warp = (nvec + 31) / 32 * 32;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  T* dx = static_cast<T*>(a.dx) + row * a.lddx;
  const float m = a.mean[row], rs = a.rstd[row];
  // xhat and g = dy w of a vector
  auto read = [&](int64_t vec, float (&xh)[V], float (&g)[V]) {
    float w[V];
    Elem<T>::unpack(load_one(x, W, vec), xh);
    Elem<T>::unpack(load_one(dy, W, vec), g);
    if (a.weight) load_f32<TW, V>(static_cast<const TW*>(a.weight), W, vec, w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      xh[e] = (xh[e] - m) * rs;
      if (a.weight) g[e] *= w[e];
    }
  };
  float c1 = 0.f, c2 = 0.f, xh[V], g[V];
  for (int64_t vec = threadIdx.x; (vec + 1) * V <= W; vec += kThreads) {
    read(vec, xh, g);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c1 += g[e];
      c2 += g[e] * xh[e];
    }
  }
  if (W % V != 0 && threadIdx.x == W / V % kThreads) {  // the row's last, partial vector
    read(W / V, xh, g);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (e < W % V) {
        c1 += g[e];
        c2 += g[e] * xh[e];
      }
    }
  }
  c1 = row_sum<kThreads>(c1, buf[0]) / static_cast<float>(W);
  c2 = row_sum<kThreads>(c2, buf[1]) / static_cast<float>(W);
  for (int64_t vec = threadIdx.x; vec < nvec_warp; vec += kThreads) {
    read(vec, xh, g);
#pragma unroll
    for (int e = 0; e < V; ++e) g[e] = rs * (g[e] - c1 - xh[e] * c2);
    store_vec(dx, W, vec, Elem<T>::pack(g));
  }
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads) layer_norm_columns_wide_kernel(LayerNormGradArgs a) {
  constexpr int V = Elem<T>::kVec;
  const int64_t W = a.width, vec = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (vec * V >= W) return;
  float sw[V], sb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sw[e] = sb[e] = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float xv[V], dy[V];
    Elem<T>::unpack(load_one(static_cast<const T*>(a.x) + row * a.ldx, W, vec), xv);
    Elem<T>::unpack(load_one(static_cast<const T*>(a.dy) + row * a.lddy, W, vec), dy);
    const float m = __ldg(a.mean + row), rs = __ldg(a.rstd + row);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sw[e] += dy[e] * ((xv[e] - m) * rs);
      sb[e] += dy[e];
    }
  }
  float* part = a.partial + int64_t(blockIdx.y) * 2 * W;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (vec * V + e < W) {
      part[vec * V + e] = sw[e];
      part[W + vec * V + e] = sb[e];
    }
}

// dweight and dbias from the partial sums: 32 columns and 32 row lanes per
// block, each lane adding every 32nd group in order, then the lanes in order.
template <typename TW>
__global__ void __launch_bounds__(1024) layer_norm_reduce_kernel(const float* partial, int groups,
                                                                 int64_t W, TW* dweight, TW* dbias) {
  __shared__ float s[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  TW* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const int64_t c = int64_t(blockIdx.x) * 32 + tx;
  float v = 0.f;
  if (c < W) {
    const float* p = partial + int64_t(blockIdx.y) * W + c;
#pragma unroll 5
    for (int g = ty; g < groups; g += 32) v += __ldg(p + int64_t(g) * 2 * W);
  }
  s[ty][tx] = v;
  __syncthreads();
  if (ty == 0 && c < W) {
    v = s[0][tx];
#pragma unroll
    for (int i = 1; i < 32; ++i) v += s[i][tx];
    out[c] = Elem<TW>::from_float(v);
  }
}

// Blocks of a launch are counted for a GB300's 152 SMs, as constants: the order
// of the sums over rows does not depend on the device.
constexpr int64_t kSms = 152;
// Up to this many rows the backward pass is one launch that reads x and dy
// twice: 64 rows of 1024, 4096, 16384 columns take 3.5, 4.2, 7.0 us (f32) and
// 3.8, 4.4, 8.1 us (bf16), where 65 take the persistent blocks and the reduction
// 4.8, 7.3, 20.8 us and 5.4, 9.2, 28.5 us.  A call that wants dx alone takes the
// same launch at any number of rows, for its blocks of one row: faster than the
// persistent blocks with their sums at 1000 x 1024 (f32 5.2 us for 10.2, bf16 4.5
// for 12.4) and slower where the ring pays, f32 8192 x 4096 78 us for 51, bf16 64
// for 45.  (A form of the persistent blocks without sums is not there.)
constexpr int64_t kFewRows = 64;

// More than 48 KB of shared memory, static included, has to be asked for once
// per device.
template <typename K, typename... Args>
cudaError_t launch(PerDeviceOnce& once, K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   Args... args) {
  if (smem > 32 * 1024) {
    const cudaError_t e = once.run([&](int) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    });
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, threads, smem, stream>>>(args...);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename TW, int kThreads, int kTpr, int kElems>
cudaError_t launch_forward(const LayerNormArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once, once_plain;
  constexpr size_t kSmem = size_t(kStages) * kElems * sizeof(T) * kThreads;
  const int64_t work = (a.rows + kThreads / kTpr - 1) / (kThreads / kTpr);
  const int64_t most = forward_blocks(kThreads, kElems) * kSms;
  const dim3 grid(static_cast<unsigned>(work < most ? work : most));
  if (plain_rows<T>(a.x, a.ldx, a.rows, a.width) && plain_rows<T>(a.y, a.ldy, a.rows, a.width))
    return launch(once_plain, layer_norm_forward_kernel<T, TW, kThreads, kTpr, kElems, true>, grid, kThreads, kSmem,
                  stream, a);
  return launch(once, layer_norm_forward_kernel<T, TW, kThreads, kTpr, kElems, false>, grid, kThreads, kSmem, stream,
                a);
}

template <typename T, typename TW>
cudaError_t forward(const LayerNormArgs& a, cudaStream_t stream) {
  const int64_t W = a.width;
  if (W <= 512) return launch_forward<T, TW, 256, 32, 16>(a, stream);
  if (W <= 2048) return launch_forward<T, TW, 128, 128, 16>(a, stream);
  if (W <= 4096) return launch_forward<T, TW, 256, 256, 16>(a, stream);
  if (W <= 8192) return launch_forward<T, TW, 256, 256, 32>(a, stream);
  if (W <= 16384) return launch_forward<T, TW, 512, 512, 32>(a, stream);
  layer_norm_forward_wide_kernel<T, TW, 1024><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

template <typename T, typename TW, int kThreads, int kTpr, int kDepth>
cudaError_t launch_backward(const LayerNormGradArgs& a, int groups, cudaStream_t stream) {
  constexpr size_t kStage = size_t(2) * kElems * sizeof(T) * kThreads;
  static PerDeviceOnce once, once_plain, once_few;
  if (groups > 0) {
    if (plain_rows<T>(a.x, a.ldx, a.rows, a.width) && plain_rows<T>(a.dy, a.lddy, a.rows, a.width) &&
        (!a.dx || plain_rows<T>(a.dx, a.lddx, a.rows, a.width)))
      return launch(once_plain, layer_norm_backward_kernel<T, TW, kThreads, kTpr, kDepth, true>, dim3(groups),
                    kThreads, kDepth * kStage, stream, a);
    return launch(once, layer_norm_backward_kernel<T, TW, kThreads, kTpr, kDepth, false>, dim3(groups), kThreads,
                  kDepth * kStage, stream, a);
  }
  const int64_t row_blocks = a.dx ? (a.rows + kThreads / kTpr - 1) / (kThreads / kTpr) : 0;
  const int64_t column_blocks = a.dweight || a.dbias ? (a.width + kThreads - 1) / kThreads : 0;
  return launch(once_few, layer_norm_backward_few_kernel<T, TW, kThreads, kTpr>,
                dim3(static_cast<unsigned>(row_blocks + column_blocks)), kThreads, kStage, stream, a,
                static_cast<int>(row_blocks));
}

template <typename T, typename TW>
cudaError_t backward(LayerNormGradArgs a, cudaStream_t stream) {
  constexpr int V = Elem<T>::kVec;
  const int64_t W = a.width;
  const bool sums = a.dweight != nullptr || a.dbias != nullptr;
  const bool wide = W > 16384, few = !wide && (a.rows <= kFewRows || !sums);
  const int64_t most = W <= 512 ? 2 * kSms : W <= 2048 ? 4 * kSms : W <= 4096 ? 2 * kSms : kSms;
  const int64_t work = W <= 512 ? (a.rows + 7) / 8 : a.rows;
  const int groups = few ? 0 : static_cast<int>(work < most ? work : most);
  float* partial = nullptr;
  if (sums && !few) {
    const cudaError_t e = pool_alloc(reinterpret_cast<void**>(&partial),
                                     size_t(groups) * 2 * W * sizeof(float), stream);
    if (e != cudaSuccess) return e;
  }
  a.partial = partial;
  cudaError_t e = cudaSuccess;
  if (wide) {
    if (a.dx) {
      layer_norm_dx_wide_kernel<T, TW, 1024><<<static_cast<unsigned>(a.rows), 1024, 0, stream>>>(a);
      note_launch();
      e = cudaGetLastError();
    }
    if (sums && e == cudaSuccess) {
      const unsigned gx = static_cast<unsigned>(((W + V - 1) / V + 255) / 256);
      layer_norm_columns_wide_kernel<T, 256><<<dim3(gx, groups), 256, 0, stream>>>(a);
      note_launch();
      e = cudaGetLastError();
    }
  } else if (W <= 512) {
    e = launch_backward<T, TW, 256, 32, 3>(a, groups, stream);
  } else if (W <= 2048) {
    e = launch_backward<T, TW, 128, 128, 3>(a, groups, stream);
  } else if (W <= 4096) {
    e = launch_backward<T, TW, 256, 256, 3>(a, groups, stream);
  } else if (W <= 8192) {
    e = launch_backward<T, TW, 512, 512, 3>(a, groups, stream);
  } else {
    // (f32: one stage is 128 KB)
    e = launch_backward<T, TW, 1024, 1024, sizeof(T) == 4 ? 1 : 3>(a, groups, stream);
  }
  if (partial == nullptr) return e;
  if (e == cudaSuccess) {
    layer_norm_reduce_kernel<TW><<<dim3(static_cast<unsigned>((W + 31) / 32), 2), 1024, 0, stream>>>(
        partial, groups, W, static_cast<TW*>(a.dweight), static_cast<TW*>(a.dbias));
    note_launch();
    e = cudaGetLastError();
  }
  const cudaError_t f = cudaFreeAsync(partial, stream);
  return e != cudaSuccess ? e : f;
}

// Without rows the weight's gradients are zero.
template <typename TW>
cudaError_t zero_grads(const LayerNormGradArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (a.dweight) e = cudaMemsetAsync(a.dweight, 0, size_t(a.width) * sizeof(TW), stream);
  if (a.dbias && e == cudaSuccess) e = cudaMemsetAsync(a.dbias, 0, size_t(a.width) * sizeof(TW), stream);
  return e;
}

}  // namespace

cudaError_t launch_layer_norm_forward(const LayerNormArgs& a, cudaStream_t stream) {
  if (a.rows == 0 || a.width == 0) return cudaSuccess;
  if (!a.bf16) return forward<float, float>(a, stream);
  return a.weight_bf16 ? forward<bf16, bf16>(a, stream) : forward<bf16, float>(a, stream);
}

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, cudaStream_t stream) {
  if (a.width == 0) return cudaSuccess;
  if (a.rows == 0) return a.weight_bf16 ? zero_grads<bf16>(a, stream) : zero_grads<float>(a, stream);
  if (!a.dx && !a.dweight && !a.dbias) return cudaSuccess;
  if (!a.bf16) return backward<float, float>(a, stream);
  return a.weight_bf16 ? backward<bf16, bf16>(a, stream) : backward<bf16, float>(a, stream);
}

}  // namespace det
