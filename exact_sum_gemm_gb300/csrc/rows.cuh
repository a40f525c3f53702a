// Row access for the row-wise training operators (layer norm, token log
// probabilities): 16-byte logical vectors of a row that may start at any
// element, block-wide reductions in a fixed order, and the element types.
//
// The i-th vector of a row always holds elements i*kVec .. i*kVec + kVec - 1,
// wherever the row lies in memory, and threads are assigned vectors by that
// index alone: a row's sums are taken in the same order, and give the same
// bits, at any address, stride or number of rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace det {

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;                       // elements per 16 bytes
  static constexpr uint32_t kNegInf = 0xFF800000u;     // a word of -inf elements
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};

// Bytes mis .. mis + 15 of the 32 bytes (lo, hi); 0 < mis < 16, mis even.
__device__ __forceinline__ uint4 shift_pair(const uint4& lo, const uint4& hi, uint32_t mis) {
  uint32_t w0 = lo.x, w1 = lo.y, w2 = lo.z, w3 = lo.w, w4 = hi.x, w5 = hi.y, w6 = hi.z, w7 = hi.w;
  if (mis & 8u) {
    w0 = w2, w1 = w3, w2 = w4, w3 = w5, w4 = w6, w5 = w7;
  }
  if (mis & 4u) {
    w0 = w1, w1 = w2, w2 = w3, w3 = w4, w4 = w5;
  }
  if (mis & 2u) {
    w0 = __funnelshift_r(w0, w1, 16);
    w1 = __funnelshift_r(w1, w2, 16);
    w2 = __funnelshift_r(w2, w3, 16);
    w3 = __funnelshift_r(w3, w4, 16);
  }
  return make_uint4(w0, w1, w2, w3);
}

// Vector `vec` of the row of n elements at p, element by element; elements
// past the end read as the halves/words of `fill`.
template <typename T>
__device__ __forceinline__ uint4 load_vec_elems(const T* p, int64_t n, int64_t vec, uint32_t fill) {
  constexpr int V = Elem<T>::kVec;
  const int64_t i = vec * V;
  uint32_t w[4] = {fill, fill, fill, fill};
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if (i + e < n) {
      if (sizeof(T) == 4) {
        w[e & 3] = __ldg(reinterpret_cast<const uint32_t*>(p) + i + e);
      } else {
        const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(p) + i + e);
        w[e / 2] = (e & 1) ? ((w[e / 2] & 0xFFFFu) | (h << 16)) : ((w[e / 2] & 0xFFFF0000u) | h);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Vectors vec0, vec0 + stride, ... of the row of n elements at p, kVpt of them.
// A row that starts off a 16-byte boundary is read as the two aligned granules
// around each vector (the second is the next lane's first, so it comes from
// L1) and shifted.  Every load is issued before any is used; what reaches
// outside the row is never touched, its vectors are read by elements.
template <typename T, int kVpt>
__device__ __forceinline__ void load_vecs(const T* p, int64_t n, int64_t vec0, int64_t stride, uint32_t fill,
                                          uint4 (&r)[kVpt]) {
  constexpr int V = Elem<T>::kVec;
  const uintptr_t row = reinterpret_cast<uintptr_t>(p);
  const uint32_t mis = static_cast<uint32_t>(row & 15u);
  if (mis == 0) {
#pragma unroll
    for (int i = 0; i < kVpt; ++i) {
      const int64_t vec = vec0 + i * stride;
      r[i] = make_uint4(fill, fill, fill, fill);
      if ((vec + 1) * V <= n) r[i] = __ldg(reinterpret_cast<const uint4*>(row) + vec);
    }
    if (n % V != 0) {                                   // the row's last, partial vector
#pragma unroll
      for (int i = 0; i < kVpt; ++i)
        if (vec0 + i * stride == n / V) r[i] = load_vec_elems(p, n, n / V, fill);
    }
    return;
  }
  // granule g of the row lies at row - mis + 16 g; those in [1, last) are whole
  const uint4* granule = reinterpret_cast<const uint4*>(row - mis);
  const int64_t last = (static_cast<int64_t>(mis) + n * static_cast<int64_t>(sizeof(T))) / 16;
  uint4 hi[kVpt];
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    const int64_t vec = vec0 + i * stride;
    r[i] = hi[i] = make_uint4(fill, fill, fill, fill);
    if (vec >= 1 && vec < last) r[i] = __ldg(granule + vec);
    if (vec + 1 < last) hi[i] = __ldg(granule + vec + 1);
  }
#pragma unroll
  for (int i = 0; i < kVpt; ++i) {
    const int64_t vec = vec0 + i * stride;
    r[i] = shift_pair(r[i], hi[i], mis);
    if (vec * V < n && (vec < 1 || vec + 1 >= last)) r[i] = load_vec_elems(p, n, vec, fill);
  }
}

// ------------------------------------------------------------ private ring
// Each thread copies its vectors of the rows to come into 16-byte slots of
// shared memory of its own, with cp.async, and reads them back itself: the
// loads are in flight without holding registers, and no barrier is needed.
// Slot i of thread t lies at base + 16 (i * threads + t).
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void ring_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
// kPlain: the row starts on a 16-byte boundary and is whole vectors; slots past
// its end are then left as they are.
template <typename T, int kVpt, bool kPlain>
__device__ __forceinline__ void ring_load(uint4* slots, int threads, const T* p, int64_t n, int64_t vec0,
                                          int64_t stride, uint32_t fill) {
  constexpr int V = Elem<T>::kVec;
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
  if constexpr (kPlain) {
    const uint4* from = reinterpret_cast<const uint4*>(p) + vec0;
    const int64_t left = n / V - vec0;
#pragma unroll
    for (int i = 0; i < kVpt; ++i)
      if (i * stride < left)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * threads * 16),
                     "l"(from + i * stride)
                     : "memory");
  } else {
    uint4 r[kVpt];
    load_vecs<T, kVpt>(p, n, vec0, stride, fill, r);
#pragma unroll
    for (int i = 0; i < kVpt; ++i) slots[i * threads] = r[i];
  }
}
// Whether rows at p, p + ld, ... of n elements are plain.
template <typename T>
inline bool plain_rows(const void* p, int64_t ld, int64_t rows, int64_t n) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && n % Elem<T>::kVec == 0 &&
         (rows <= 1 || ld % Elem<T>::kVec == 0);
}

// Elements [from, to) of the vector v to p[0 ..].
template <typename T>
__device__ __forceinline__ void store_elems(T* at, const uint4& v, int from, int to) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < Elem<T>::kVec; ++e) {
    if (e >= from && e < to) {
      if (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(at)[e] = w[e & 3];
      } else {
        reinterpret_cast<uint16_t*>(at)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
      }
    }
  }
}

// Writes vector `vec` of the row of n elements at p.  Called by whole warps
// whose lane l holds vector vec(lane 0) + l.  A row off a 16-byte boundary is
// written in aligned granules put together from neighbouring lanes' vectors;
// the warp's two edges and the row's last, partial vector go element by
// element.
template <typename T>
__device__ __forceinline__ void store_vec(T* p, int64_t n, int64_t vec, const uint4& v) {
  constexpr int V = Elem<T>::kVec;
  const int64_t i = vec * V;
  T* at = p + i;
  const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 15u);
  const bool full = i + V <= n;
  if (mis == 0) {
    if (full) {
      *reinterpret_cast<uint4*>(at) = v;
    } else if (i < n) {
      store_elems(at, v, 0, static_cast<int>(n - i));
    }
    return;
  }
  const int lane = threadIdx.x & 31;
  uint4 next;
  next.x = __shfl_down_sync(0xFFFFFFFFu, v.x, 1);
  next.y = __shfl_down_sync(0xFFFFFFFFu, v.y, 1);
  next.z = __shfl_down_sync(0xFFFFFFFFu, v.z, 1);
  next.w = __shfl_down_sync(0xFFFFFFFFu, v.w, 1);
  if (i >= n) return;
  if (!full) {
    store_elems(at, v, 0, static_cast<int>(n - i));
    return;
  }
  const int head = static_cast<int>((16u - mis) / sizeof(T));  // elements before the boundary
  if (lane == 0) store_elems(at, v, 0, head);
  if (lane < 31 && i + 2 * V <= n) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(at) + (16u - mis)) =
        shift_pair(v, next, 16u - mis);
  } else {
    store_elems(at, v, head, V);
  }
}

// Elements d .. d + 7 of a row of `dim`, 0 past its end.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int d, int dim, float (&f)[8]) {
  constexpr int V = Elem<T>::kVec;
  if (d + 8 <= dim && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
    for (int v = 0; v < 8 / V; ++v) {
      float x[V];
      Elem<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p + d) + v), x);
#pragma unroll
      for (int e = 0; e < V; ++e) f[v * V + e] = x[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = d + e < dim ? Elem<T>::to_float(p[d + e]) : 0.f;
  }
}
__device__ __forceinline__ float dot8(const float (&x)[8], const float (&y)[8]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Maximum and minimum that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// 2^x (2 ulp; 0 below the normal range).
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A probability from its binary logarithm, which is at most 0 but for the
// rounding of what it is the difference of.
__device__ __forceinline__ float probability(float x) { return exp2_approx(min_nan(x, 0.f)); }

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace det
