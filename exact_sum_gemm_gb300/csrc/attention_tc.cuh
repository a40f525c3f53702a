// Building blocks of the tensor-core attention kernels: tiles and their
// products, TMA and cp.async loads, the split of f32 into bf16 planes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "det_train.h"
#include "rows.cuh"
#include "tc_ptx.cuh"

namespace det {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();          // gemm_tc.cu

namespace {

// Head dimensions up to this fit the f32 kernels with one panel a plane; larger
// ones take the kernels of attention_wide.cu.
constexpr int kNarrowDim = 64;

typedef __nv_bfloat16 bf16;

constexpr int kLoaders = 64;
constexpr int kThreads = 384;                           // (12 warps leave a thread 168 registers)
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kAhead = 2;                               // items in flight per loader thread

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
  return ptx::mbar_wait_ns(bar, parity, kWaitLimitNs);
}
// Whether the phase is over, at once.
__device__ __forceinline__ bool phase_over(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred P1;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 P1, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P1;\n\t}"
      : "=r"(done)
      : "r"(ptx::smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// The same for a whole warp, which goes on together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t dst, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src)
               : "memory");
  return v;
}

// The warp's arrival, by one lane for all: 256 arrivals of threads at one
// barrier are made one after the other.
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// One thread issues the products, in loops that are unrolled so that each MMA
// costs two additions to its descriptors: a 128 x 64 x 16 product then takes 48
// cycles, which is what its operands take to be read from shared memory.  (All
// lanes going along with the issue predicated on one: 64 at least, and 75 to
// 100 with the descriptors' arithmetic.)
// D[tmem] (+)= A[tmem] B[smem]: A is 128 lanes of packed bf16 pairs.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

// A tile is [rows][64] bf16 panels, 128-byte swizzled, panel after panel.  As
// an MN-major operand (the 64 columns are its rows) the panels are the leading
// stride and 8-row groups the other.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t panel_bytes) {
  return (ptx::smem_desc_sw128(saddr) & ~(uint64_t(0x3FFF) << 16)) | (uint64_t(panel_bytes >> 4) << 16);
}
constexpr uint32_t kMnB = 1u << 16;                     // instruction descriptor: B is MN-major

__host__ __device__ constexpr uint32_t panel_bytes(int rows) { return rows * 128u; }

// The pairs of planes whose products are taken, smallest first.
__host__ __device__ constexpr int pair_count(int planes) { return planes == 3 ? 6 : 1; }
__host__ __device__ constexpr int pair_a(int planes, int i) {
  return planes == 1 ? 0 : i == 0 ? 2 : i == 1 ? 0 : i == 2 ? 1 : i == 3 ? 1 : i == 4 ? 0 : 0;
}
__host__ __device__ constexpr int pair_b(int planes, int i) {
  return planes == 1 ? 0 : i == 0 ? 0 : i == 1 ? 2 : i == 2 ? 1 : i == 3 ? 0 : i == 4 ? 1 : 0;
}

// D = A B^T over ksteps x 16 columns, both K-major: kPlanes tiles of kARows and
// kBRows rows, each of up to kPanels panels.
template <int kPlanes, int kARows, int kBRows, int kPanels>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a, uint32_t b, int ksteps,
                                           uint32_t idesc) {
  const uint64_t ad = ptx::smem_desc_sw128(a), bd = ptx::smem_desc_sw128(b);
  constexpr uint32_t kA = panel_bytes(kARows) >> 4, kB = panel_bytes(kBRows) >> 4;
#pragma unroll
  for (int i = 0; i < pair_count(kPlanes); ++i)
#pragma unroll
    for (int k = 0; k < 4 * kPanels; ++k) {
      if (k >= ksteps) break;
      // 32 bytes a step, four steps a panel
      ptx::mma_bf16(d, ad + (k & 3) * 2 + ((k >> 2) + kPanels * pair_a(kPlanes, i)) * kA,
                    bd + (k & 3) * 2 + ((k >> 2) + kPanels * pair_b(kPlanes, i)) * kB, idesc, i + k > 0);
    }
}
// D (+)= A B over kRows rows of B's tile, A packed in TMEM.  One plane: 16 words
// per 32 rows, kGap words from one 32 to the next.  Three: 8 words of the first
// and 8 of the second per 16 rows, the third at a2 without gaps.
template <int kPlanes, int kRows, int kGap, int kPanels>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t a2, uint32_t b,
                                           uint32_t idesc, bool accumulate) {
  const uint64_t bd = desc_mn(b, panel_bytes(kRows));
#pragma unroll
  for (int i = 0; i < pair_count(kPlanes); ++i) {
    const int plane = pair_a(kPlanes, i);
#pragma unroll
    for (int k = 0; k < kRows / 16; ++k)                // 16 rows are 2048 bytes
      mma_ts(d,
             kPlanes == 1 ? a + (k / 2) * kGap + (k & 1) * 8 : plane == 2 ? a2 + k * 8 : a + k * 16 + plane * 8,
             bd + k * (2048 >> 4) + kPanels * pair_b(kPlanes, i) * (panel_bytes(kRows) >> 4), idesc,
             accumulate || i + k > 0);
  }
}

// One head of a tensor as the loaders read it.
struct Source {
  const bf16* p;
  int64_t stride;
  int rows, dim, panels;
  bool vec;                                             // 16-byte pieces are aligned
};
__device__ __forceinline__ Source source(const Heads& h, int batch, int head, int rows, int dim) {
  Source s;
  s.p = static_cast<const bf16*>(h.p) + int64_t(batch) * h.sb + int64_t(head) * h.sh;
  s.stride = h.sl;
  s.rows = rows;
  s.dim = dim;
  s.panels = dim > 64 ? 2 : 1;
  s.vec = dim % 8 == 0 && h.sl % 8 == 0 && (reinterpret_cast<uintptr_t>(s.p) & 15u) == 0;
  return s;
}

// The tensor maps of a launch.
struct Maps {
  CUtensorMap m[4];
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y,
                                            int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// kRows rows of a head into their panels; of three planes (entries batch,
// batch + batches, ... of the map), one after the other.
template <int kPlanes, int kRows>
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int panels, int row0,
                                         int head, int batch, int batches) {
  if constexpr (kPlanes == 1) {
    for (int p = 0; p < panels; ++p)
      tma_load_4d(dst + p * panel_bytes(kRows), map, bar, 64 * p, row0, head, batch);
  } else {
    for (int p = 0; p < kPlanes * panels; ++p) {
      const int plane = p / panels, panel = p - plane * panels;
      tma_load_4d(dst + p * panel_bytes(kRows), map, bar, 64 * panel, row0, head, batch + plane * batches);
    }
  }
}
// `bytes` (a multiple of 16, both sides aligned) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   ptx::smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_addr(bar))
               : "memory");
}

// The loader thread's share of a tile: its 16-byte column c of rows r0,
// r0 + step, ...; step is 8, or 4 where there are two panels, and then the
// swizzled column of every other row differs in one bit.
struct Share {
  int c, r0, step;
  uint32_t off, flip;
};
template <int kRows>
__device__ __forceinline__ Share share_of(const Source& s, int tid) {
  const int bits = s.panels == 2 ? 4 : 3;
  Share h;
  h.c = tid & ((1 << bits) - 1);
  h.r0 = tid >> bits;
  h.step = kLoaders >> bits;
  h.off = (h.c >> 3) * panel_bytes(kRows) + h.r0 * 128 + (((h.c & 7) ^ (h.r0 & 7)) << 4);
  h.flip = (h.step & 7) << 4;
  return h;
}

// Starts the copy of rows row0 .. row0 + kRows - 1.
template <int kRows>
__device__ __forceinline__ void load_rows(uint32_t dst, const Source& s, int row0, int tid) {
  const Share h = share_of<kRows>(s, tid);
  if (h.c * 8 >= ((s.dim + 15) & ~15)) return;          // (no product reads it)
  const int d = h.c * 8;
  uint32_t off = h.off;
  const bf16* p = s.p + int64_t(row0 + h.r0) * s.stride + d;
  if (s.vec) {
#pragma unroll 8
    for (int r = h.r0; r < kRows; r += h.step) {
      const bool valid = row0 + r < s.rows && d < s.dim;
      cp_async16(dst + off, valid ? p : s.p, valid);
      p += h.step * s.stride;
      off = (off + h.step * 128) ^ h.flip;
    }
  } else {
    for (int r = h.r0; r < kRows; r += h.step) {
      uint32_t w[4] = {0, 0, 0, 0};
      if (row0 + r < s.rows) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (d + i < s.dim) w[i / 2] |= uint32_t(e[i]) << (16 * (i & 1));
      }
      sts128(dst + off, make_uint4(w[0], w[1], w[2], w[3]));
      p += h.step * s.stride;
      off = (off + h.step * 128) ^ h.flip;
    }
  }
}

// The top bits of the non-finite halves: one whose exponent is all ones carries
// into its top bit.
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + 0x00800080u) & 0x80008000u;
}

// The thread's share of a loaded tile of rows row0 ..: rows at or past the end
// become zero (unless they are, past_zero) and, where asked, non-finite values;
// whether there were any.
template <int kRows>
__device__ __forceinline__ bool clean_rows(uint32_t dst, const Source& s, int row0, bool past_zero, bool finite,
                                           int tid) {
  const Share h = share_of<kRows>(s, tid);
  if (h.c * 8 >= ((s.dim + 15) & ~15)) return false;
  if (past_zero || row0 + kRows <= s.rows) {
    // look first, eight loads at a time: as a rule there is nothing to do
    uint32_t off = h.off, any = 0;
    for (int r = h.r0; r < kRows; r += 8 * h.step) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i, off = (off + h.step * 128) ^ h.flip) v[i] = lds128(dst + off);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        any |= non_finite(v[i].x) | non_finite(v[i].y) | non_finite(v[i].z) | non_finite(v[i].w);
    }
    if (any == 0) return false;
  }
  bool found = false;
  uint32_t off = h.off;
  for (int r = h.r0; r < kRows; r += h.step, off = (off + h.step * 128) ^ h.flip) {
    const uint32_t at = dst + off;
    if (row0 + r >= s.rows) {
      sts128(at, make_uint4(0, 0, 0, 0));
    } else if (finite) {
      uint4 v = lds128(at);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      bool any = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t top = non_finite(w[i]);
        if (top & 0x80000000u) w[i] &= 0x0000FFFFu, any = true;
        if (top & 0x00008000u) w[i] &= 0xFFFF0000u, any = true;
      }
      if (any) sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
      found |= any;
    }
  }
  return found;
}

__device__ __forceinline__ void report_timeout(unsigned* status) {
  if (status != nullptr) atomicOr(status, kStatusTimeout);
}

template <bool kMin>
__device__ __forceinline__ float extreme3(float a, float b, float c) {
  float r;
  if (kMin) asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  else asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two f32 values as packed bf16 pairs: kPlanes words whose sum they are (three)
// or are rounded to (one).
template <int kPlanes>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&w)[kPlanes]) {
#pragma unroll
  for (int p = 0; p < kPlanes; ++p) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w[p] = *reinterpret_cast<const uint32_t*>(&h);
    if (p + 1 < kPlanes) {
      x -= __uint_as_float(w[p] << 16);
      y -= __uint_as_float(w[p] & 0xFFFF0000u);
    }
  }
}

// 16 f32 values, in columns at `to`, as three planes: the first two over them,
// the third at `third`.
__device__ __forceinline__ void put_planes(const uint32_t (&x)[16], uint32_t to, uint32_t third) {
  uint32_t w[3][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t part[3];
    split_pair<3>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), part);
    w[0][e] = part[0], w[1][e] = part[1], w[2][e] = part[2];
  }
  tmem_st8(to, w[0]);
  tmem_st8(to + 8, w[1]);
  tmem_st8(third, w[2]);
}
// sum += the columns at taddr.
template <int N>
__device__ __forceinline__ void add_columns(float (&sum)[N], uint32_t taddr) {
#pragma unroll
  for (int cb = 0; cb < N; cb += 32) {
    uint32_t v[32];
    ptx::tmem_ld32(taddr + cb, v);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) sum[cb + e] += __uint_as_float(v[e]);
  }
}

__device__ __forceinline__ void store_columns(float* p, int d0, int dim, const uint32_t (&v)[32], float by) {
  if (dim % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (d0 + 4 * c < dim)
        *reinterpret_cast<float4*>(p + d0 + 4 * c) =
            make_float4(__uint_as_float(v[4 * c]) * by, __uint_as_float(v[4 * c + 1]) * by,
                        __uint_as_float(v[4 * c + 2]) * by, __uint_as_float(v[4 * c + 3]) * by);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (d0 + e < dim) p[d0 + e] = __uint_as_float(v[e]) * by;
  }
}
// Row `row` of a head from 32 accumulator columns at column d0, times `by`.
__device__ __forceinline__ void store_columns(bf16* p, int d0, int dim, const uint32_t (&v)[32], float by) {
  if (dim % 8 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (d0 + 8 * c < dim) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(v[8 * c + e]) * by;
        *reinterpret_cast<uint4*>(p + d0 + 8 * c) = Elem<bf16>::pack(f);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (d0 + e < dim) p[d0 + e] = __float2bfloat16_rn(__uint_as_float(v[e]) * by);
  }
}

__device__ __forceinline__ int keys_of(const AttentionArgs& a, int batch) {
  return a.k_lengths ? max(0, min(a.lk, __ldg(a.k_lengths + batch))) : a.lk;
}

// Scores at or past column `seen`: infinite, of the sign that the scale takes
// to -inf.
__device__ __forceinline__ void hide(uint32_t (&v)[32], int seen, float scale) {
  const uint32_t hidden = scale < 0.f ? 0x7F800000u : 0xFF800000u;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (e >= seen) v[e] = hidden;
}

// 2^(s c - ref) is taken with one rounding, ref being the rounded s c of some s.
// Its rounding is a factor of all of a row's exponentials, which cancels while it
// is small: below kFar at most 2^(2^-11), so that the largest probability is 1
// rounded to bf16 too; from 2^30 on they would overflow.  Further away the scores
// are multiplied and rounded as ref was.
constexpr float kFar = 8192.f;
__device__ __forceinline__ void scale_far(uint32_t (&v)[32], float ref, float c) {
  const float by = fabsf(ref) >= kFar ? c : 1.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), by));
}

// Maximum (minimum) of a row's scores; NaN if one is.
template <bool kMin>
__device__ __forceinline__ float row_extreme(const uint32_t (&v)[2][32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t(&x)[32] = v[i / 2];
    const int e0 = 16 * (i & 1);
    m[i] = __uint_as_float(x[e0 + 15]);
#pragma unroll
    for (int e = 0; e < 14; e += 2)
      m[i] = extreme3<kMin>(m[i], __uint_as_float(x[e0 + e]), __uint_as_float(x[e0 + e + 1]));
    m[i] = extreme3<kMin>(m[i], m[i], __uint_as_float(x[e0 + 14]));
  }
  return extreme3<kMin>(extreme3<kMin>(m[0], m[1], m[2]), m[3], m[3]);
}

// Tensor map of a [batch, length, heads, dim] tensor in boxes of 64 columns and
// `rows` rows of one head; false where the tensor is not one that TMA reads.
inline bool make_map(CUtensorMap* map, const Heads& t, int64_t batch, int64_t length, int64_t heads, int64_t dim,
              int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr || (reinterpret_cast<uintptr_t>(t.p) & 15u) != 0) return false;
  const cuuint64_t dims[4] = {cuuint64_t(dim), cuuint64_t(length), cuuint64_t(heads), cuuint64_t(batch)};
  const int64_t elements[3] = {t.sl, t.sh, t.sb};
  cuuint64_t strides[3];
  for (int i = 0; i < 3; ++i) {
    // (the stride of an axis of one is never used)
    const int64_t s = dims[i + 1] == 1 ? 64 : elements[i];
    if (dims[i + 1] == 0 || s <= 0 || s % 8 != 0 || s >= (int64_t(1) << 38)) return false;
    strides[i] = cuuint64_t(s) * 2;
  }
  const cuuint32_t box[4] = {64, cuuint32_t(rows), 1, 1}, ones[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t.p, dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Planes of a tensor in scratch: [plane][batch][heads][length][width].
inline Heads planes_of(void* p, int64_t length, int64_t heads, int64_t width) {
  return {p, heads * length * width, width, length * width};
}

}  // namespace
}  // namespace det
