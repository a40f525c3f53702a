// f32 attention on the tensor cores for head dimensions of 65 to 128.
//
// The formulas and the three bf16 planes are those of attention_tc.cu; what is
// different is that 128 rows of two operands in three planes do not fit shared
// memory at this dimension.
//
// Forward: a block owns 128 queries (96 KB of planes) and goes over the keys 64
// at a time.  The two softmax groups share the rows, 32 columns of S each; they
// exchange their maxima through shared memory, and each sums 64 columns of O.
//
// Backward: a block owns 64 keys (queries).  Its K and V (Q and dO) are stacked
// as the 128 rows of one operand A, so A Q^T holds S^T in its upper 64 rows and
// A dO^T holds dP^T in its lower 64; the other halves are not used.  The threads
// of the upper rows take P, hand it to those of the lower rows through shared
// memory, and [P; dS] is the stacked operand of the sums: its product with dO
// has dv in the upper rows, that with Q has dk in the lower.  Half of the
// tensor cores' work is thrown away, which leaves them several times faster
// than the CUDA cores all the same (f32 4 x 1024, 16 heads of 96, causal,
// forward + backward: 0.89 ms against 3.04 ms).  Steps are 32 rows.
#include "attention_tc.cuh"

namespace det {
namespace {

constexpr int kPanels = 2;
constexpr int kStages = 2;                              // tiles (or step pairs) on their way or in use
constexpr uint32_t kPlane128 = kPanels * panel_bytes(128);   // 32 KB: a plane of 128 rows

// ------------------------------------------------------------------ forward
constexpr int kKeys = 64;
constexpr uint32_t kTileBytes = 3 * kPanels * panel_bytes(kKeys);

struct ForwardShared {
  float top[2][2][128];                                 // by step parity and group
  float sum[2][128];
  uint64_t q_full, full[kStages], empty[kStages], s_full[2], p_full[2], o_done[2], drained;
  uint32_t tmem;
};

// Barrier `id` of `threads` threads.
__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    attention_wide_forward_kernel(AttentionArgs a, unsigned* status, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ ForwardShared bars;
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u, ring = base + 3 * kPlane128;
  const int tiles = (a.lq + 127) / 128;
  const int64_t rest = blockIdx.x / a.hq;
  const int h = static_cast<int>(blockIdx.x - rest * a.hq), b = static_cast<int>(rest / tiles);
  const int tile = tiles - 1 - static_cast<int>(rest - int64_t(b) * tiles);
  const int hk = h / (a.hq / a.hkv), i0 = tile * 128;
  const int keys = keys_of(a, b), offset = a.lk - a.lq, ksteps = (a.dim + 15) / 16;
  int end = keys;
  if (a.causal) end = max(0, min(end, min(i0 + 128, a.lq) + offset));
  const int n = (end + kKeys - 1) / kKeys;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars.q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars.full[s], 1);
      ptx::mbar_init(&bars.empty[s], 1);
    }
    for (int u = 0; u < 2; ++u) {
      ptx::mbar_init(&bars.s_full[u], 1);
      ptx::mbar_init(&bars.p_full[u], 8);
      ptx::mbar_init(&bars.o_done[u], 1);
    }
    ptx::mbar_init(&bars.drained, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 10) {
    ptx::tmem_alloc(&bars.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem;       // S at 64 u, the third plane of P at 128 + 32 u, O at 256

  if (warp == 8) {
    if (lane == 0 && n > 0) {
      ptx::mbar_arrive_expect_tx(&bars.q_full, 3 * kPlane128);
      tma_rows<3, 128>(base, &maps.m[0], &bars.q_full, kPanels, i0, h, b, a.batch);
      bool ok = true;
      int it = 0;                                       // K and V of every key tile in turn
      for (; it < 2 * n; ++it) {
        const int s = it % kStages;
        if (!wait_bounded(&bars.empty[s], ((it / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bars.full[s], kTileBytes);
        tma_rows<3, kKeys>(ring + s * kTileBytes, &maps.m[1 + (it & 1)], &bars.full[s], kPanels, it / 2 * kKeys, hk, b,
                           a.batch);
      }
      // nothing in flight at the block's end, however it comes
      if (!wait_bounded(&bars.q_full, 0)) ok = false;
      for (int j = max(0, it - kStages); j < it; ++j)
        if (!wait_bounded(&bars.full[j % kStages], (j / kStages) & 1)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp == 10) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, kKeys);
      bool ok = wait_bounded(&bars.q_full, 0);
      for (int j = 0; j < n && ok; ++j) {
        const int item = 2 * j, s = item % kStages;
        ok = wait_bounded(&bars.full[s], (item / kStages) & 1);
        // (P of the step before the last is where S goes)
        if (ok && j >= 2) ok = wait_bounded(&bars.o_done[j & 1], ((j >> 1) - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        product_ss<3, 128, kKeys, kPanels>(tmem + 64 * (j & 1), base, ring + s * kTileBytes, ksteps, idesc);
        ptx::mma_commit(&bars.s_full[j & 1]);
        if (item + kStages < 2 * n) ptx::mma_commit(&bars.empty[s]);
      }
      if (!ok) report_timeout(status);
    }
  } else if (warp == 11) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, ksteps * 16) | kMnB;
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        const int item = 2 * j + 1, s = item % kStages;
        ok = wait_bounded(&bars.full[s], (item / kStages) & 1);
        if (ok) ok = wait_bounded(&bars.p_full[j & 1], (j >> 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        product_ts<3, kKeys, 16, kPanels>(tmem + 256, tmem + 64 * (j & 1), tmem + 128 + 32 * (j & 1),
                                          ring + s * kTileBytes, idesc, false);
        ptx::mma_commit(&bars.o_done[j & 1]);
        if (item + kStages < 2 * n) ptx::mma_commit(&bars.empty[s]);
      }
      ptx::mma_commit(&bars.drained);
      if (!wait_bounded(&bars.drained, 0)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp < 8) {
    const int w = warp >> 2, row = 32 * (warp & 3) + lane, i = i0 + row;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_at = tmem + lanes + 256 + 64 * w;  // the group's 64 columns of O
    const float c = a.scale * kLog2e;
    const int last = a.causal ? min(keys, i + offset + 1) : keys;   // keys [0, last) are visible
    float ref = -INFINITY, l = 0.f, o_sum[64];
#pragma unroll
    for (float& x : o_sum) x = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      // (a warp whose wait runs out waits no more but goes on, so that the others are not left at the
      // barriers)
      if (ok) ok = wait_warp(&bars.s_full[j & 1], (j >> 1) & 1);
      ptx::tc_fence_after();
      const uint32_t s_at = tmem + lanes + 64 * (j & 1) + 32 * w;
      const int seen = last - j * kKeys - 32 * w;       // of the group's 32 columns
      const bool whole = __all_sync(0xFFFFFFFFu, seen >= 32);
      uint32_t v[32];
      ptx::tmem_ld32(s_at, v);
      ptx::tmem_wait_ld();
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        top = max_nan(top, whole || e < seen ? __uint_as_float(v[e]) * c : -INFINITY);
      bars.top[j & 1][w][row] = top;
      named_barrier(1, 256);
      top = max_nan(top, bars.top[j & 1][w ^ 1][row]);
      const bool grow = top > ref + 8.0f || (ref == -INFINITY && top != -INFINITY);
      float by = 1.0f;
      if (grow) {
        by = exp2_approx(ref - top);
        l *= by;
        ref = top;
      }
      const float sub = ref == -INFINITY ? 0.f : ref;
      float by_c = c;
      if (__any_sync(0xFFFFFFFFu, fabsf(sub) >= kFar)) {
        scale_far(v, sub, c);
        if (fabsf(sub) >= kFar) by_c = 1.f;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float p = exp2_approx(fmaf(__uint_as_float(v[16 * g + e]), by_c, -sub));
          if (!whole && 16 * g + e >= seen) p = 0.f;
          l += p;
          x[e] = __float_as_uint(p);
        }
        put_planes(x, s_at + 16 * g, tmem + lanes + 128 + 32 * (j & 1) + 16 * w + 8 * g);
      }
      // the product of the step before has run beside this: O of it, taken with its reference,
      // joins the sum before the next product writes there
      if (j > 0) {
        if (ok) ok = wait_warp(&bars.o_done[(j - 1) & 1], ((j - 1) >> 1) & 1);
        ptx::tc_fence_after();
        add_columns(o_sum, o_at);
      }
      if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
        for (float& x : o_sum) x *= by;
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      arrive_warp(&bars.p_full[j & 1]);
    }
    if (n > 0) {
      if (ok) ok = wait_warp(&bars.o_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
      ptx::tc_fence_after();
      add_columns(o_sum, o_at);
    }
    bars.sum[w][row] = l;
    named_barrier(1, 256);
    l = bars.sum[0][row] + bars.sum[1][row];
    if (!ok && lane == 0) report_timeout(status);
    const float inv = !ok ? __uint_as_float(0x7FC00000u) : l == 0.f ? 0.f : 1.0f / l;
    if (i < a.lq) {
      float* o = static_cast<float*>(a.o.p) + int64_t(b) * a.o.sb + int64_t(h) * a.o.sh + int64_t(i) * a.o.sl;
#pragma unroll
      for (int cb = 0; cb < 64; cb += 32) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(o_sum[cb + e]);
        if (64 * w + cb < a.dim) store_columns(o, 64 * w + cb, a.dim, v, inv);
      }
      if (w == 0)
        a.lse[(int64_t(b) * a.hq + h) * a.lq + i] =
            !ok ? inv : l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 10) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ backward
constexpr int kHome = 64;                               // rows that a block owns
constexpr int kStep = 32;
constexpr uint32_t kStepBytes = 3 * kPanels * panel_bytes(kStep);
constexpr uint32_t kThird = 32, kDp = 48, kSlot = 96;   // of a slot: S or [P; dS] at 0
constexpr uint32_t kSumUpper = 256, kSumLower = 384;    // products with dO and with Q (K)

struct BackwardShared {
  alignas(16) float lse[kStages][kStep], delta[kStages][kStep];
  float p[2][kStep][kHome];                             // by step parity: P, from upper to lower rows
  uint64_t home_full, full[kStages], empty[kStages], s_full[2], p_full[2], slot_free[2], sum_full, sum_free, drained;
  uint32_t tmem;
};

// Block `block` of the keys' (kKeysHome) or of the queries'.  maps: the home
// rows' tensors (K, V or Q, dO), the steps' (Q, dO or K, V).
template <bool kKeysHome>
__device__ __forceinline__ void wide_block(const AttentionArgs& a, unsigned* status, const CUtensorMap* maps,
                                           int64_t block, unsigned char* smem_raw, BackwardShared& bars) {
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + 3 * kPlane128;           // stages of two step tiles
  const int rows = kKeysHome ? a.lk : a.lq, heads = kKeysHome ? a.hkv : a.hq;
  const int tiles = (rows + kHome - 1) / kHome;
  const int64_t rest = block / heads;
  const int h = static_cast<int>(block - rest * heads), b = static_cast<int>(rest / tiles);
  int tile = static_cast<int>(rest - int64_t(b) * tiles);
  if (!kKeysHome) tile = tiles - 1 - tile;              // most work first under a causal mask
  const int r0 = tile * kHome, share = a.hq / a.hkv;
  const int keys = keys_of(a, b), offset = a.lk - a.lq, ksteps = (a.dim + 15) / 16;
  int first = 0, end = kKeysHome ? a.lq : keys;
  if (a.causal) {
    if (kKeysHome) first = max(0, r0 - offset) / kStep * kStep;
    else end = max(0, min(end, min(r0 + kHome, a.lq) + offset));
  }
  int per = end > first ? (end - first + kStep - 1) / kStep : 0;
  if (kKeysHome && r0 >= keys) per = 0;
  const int n = per * (kKeysHome ? share : 1);
  const int h_first = kKeysHome ? h * share : h / share;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars.home_full, 1);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars.full[s], 1);
      ptx::mbar_init(&bars.empty[s], 1);
    }
    for (int u = 0; u < 2; ++u) {
      ptx::mbar_init(&bars.s_full[u], 1);
      ptx::mbar_init(&bars.p_full[u], 8);
      ptx::mbar_init(&bars.slot_free[u], 1);
    }
    ptx::mbar_init(&bars.sum_full, 1);
    ptx::mbar_init(&bars.sum_free, 8);
    ptx::mbar_init(&bars.drained, 1);
    ptx::fence_mbar_init();
  }
  if (warp == 10) {
    ptx::tmem_alloc(&bars.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars.tmem;

  if (warp == 8) {
    if (lane == 0 && n > 0) {
      ptx::mbar_arrive_expect_tx(&bars.home_full, 3 * kPlane128);
      for (int p = 0; p < 3 * kPanels; ++p) {           // the second operand's rows under the first's
        const int plane = p / kPanels, x = 64 * (p % kPanels);
        const uint32_t at = base + p * panel_bytes(128);
        tma_load_4d(at, &maps[0], &bars.home_full, x, r0, h, b + plane * a.batch);
        tma_load_4d(at + panel_bytes(kHome), &maps[1], &bars.home_full, x, r0, h, b + plane * a.batch);
      }
      bool ok = true;
      int i = 0, head = h_first, row = first;
      for (; i < n; ++i) {
        const int s = i % kStages;
        if (!wait_bounded(&bars.empty[s], ((i / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t at = ring + s * 2 * kStepBytes;
        ptx::mbar_arrive_expect_tx(&bars.full[s], 2 * kStepBytes + (kKeysHome ? 2 * kStep * 4 : 0));
        tma_rows<3, kStep>(at, &maps[2], &bars.full[s], kPanels, row, head, b, a.batch);
        tma_rows<3, kStep>(at + kStepBytes, &maps[3], &bars.full[s], kPanels, row, head, b, a.batch);
        if (kKeysHome) {
          const int64_t q = (int64_t(b) * a.hq + head) * a.stat_stride + row;
          bulk_load(bars.lse[s], a.lse2 + q, kStep * 4, &bars.full[s]);
          bulk_load(bars.delta[s], a.delta + q, kStep * 4, &bars.full[s]);
        }
        row += kStep;
        if (row >= end) {
          row = first;
          ++head;
        }
      }
      // nothing in flight at the block's end, however it comes
      if (!wait_bounded(&bars.home_full, 0)) ok = false;
      for (int j = max(0, i - kStages); j < i; ++j)
        if (!wait_bounded(&bars.full[j % kStages], (j / kStages) & 1)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp == 10) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, kStep);
      bool ok = wait_bounded(&bars.home_full, 0);
      for (int i = 0; i < n && ok; ++i) {               // S and dP of step i into its slot
        const int s = i % kStages;
        ok = wait_bounded(&bars.full[s], (i / kStages) & 1);
        if (ok && i >= 2) ok = wait_bounded(&bars.slot_free[i & 1], ((i >> 1) - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t at = ring + s * 2 * kStepBytes, d = tmem + kSlot * (i & 1);
        product_ss<3, 128, kStep, kPanels>(d, base, at, ksteps, idesc);
        product_ss<3, 128, kStep, kPanels>(d + kDp, base, at + kStepBytes, ksteps, idesc);
        ptx::mma_commit(&bars.s_full[i & 1]);
      }
      if (!ok) report_timeout(status);
    }
  } else if (warp == 11) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(128, ksteps * 16) | kMnB;
      bool ok = true;
      for (int i = 0; i < n && ok; ++i) {               // the sums, once P and dS of step i are there
        ok = wait_bounded(&bars.p_full[i & 1], (i >> 1) & 1);
        if (i > 0 && ok) ok = wait_bounded(&bars.sum_free, (i - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const int s = i % kStages;
        const uint32_t at = ring + s * 2 * kStepBytes, p = tmem + kSlot * (i & 1);
        if (kKeysHome)
          product_ts<3, kStep, 16, kPanels>(tmem + kSumUpper, p, p + kThird, at + kStepBytes, idesc, false);
        product_ts<3, kStep, 16, kPanels>(tmem + kSumLower, p, p + kThird, at, idesc, false);
        // (only where they are waited for: nothing arrives after the block's end)
        if (i + kStages < n) ptx::mma_commit(&bars.empty[s]);
        if (i + 2 < n) ptx::mma_commit(&bars.slot_free[i & 1]);
        ptx::mma_commit(&bars.sum_full);
      }
      ptx::mma_commit(&bars.drained);                   // all of the above, and S and dP before them
      if (!wait_bounded(&bars.drained, 0)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp < 8) {
    const int w = warp >> 2, at_row = 32 * (warp & 3) + lane, home = at_row & (kHome - 1), r = r0 + home;
    const bool upper = (warp & 3) < 2;                  // S and P; the others dP and dS
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float c = a.scale * kLog2e;
    float own_lse = INFINITY, own_delta = 0.f;          // of the thread's query
    if (!kKeysHome && r < a.lq) {
      const int64_t i = (int64_t(b) * a.hq + h) * a.stat_stride + r;
      own_lse = __ldg(a.lse2 + i);
      own_delta = __ldg(a.delta + i);
    }
    bool ok = true;
    int row = first + 16 * w, left = per;               // the group's first row of the step
    float total[64];                                    // 64 columns of the row's gradient
#pragma unroll
    for (float& x : total) x = 0.f;
    const bool sums = kKeysHome || !upper;
    const uint32_t total_at = tmem + lanes + (upper ? kSumUpper : kSumLower) + 64 * w;
    // P and dS of step i, 16 columns a group
    auto pairs = [&](int i) {
      // (a warp whose wait runs out waits no more but goes on, so that the others are not left at the
      // barrier; the second wait is over at once: it orders the loaded lse and delta before their use)
      if (ok) ok = wait_warp(&bars.s_full[i & 1], (i >> 1) & 1);
      if (ok && kKeysHome) ok = wait_warp(&bars.full[i % kStages], (i / kStages) & 1);
      ptx::tc_fence_after();
      const uint32_t slot = tmem + lanes + kSlot * (i & 1);
      uint32_t v[16];
      tmem_ld16(slot + (upper ? 0 : kDp) + 16 * w, v);
      // columns [lo, hi) of the 16 are visible to the thread's row
      int lo = 0, hi = 16;
      if (kKeysHome) {
        hi = a.lq - row;
        if (a.causal) lo = r - offset - row;
      } else {
        hi = keys - row;
        if (a.causal) hi = min(hi, r + offset + 1 - row);
      }
      const float* stat = (upper ? bars.lse : bars.delta)[i % kStages] + 16 * w;
      float(*p)[kHome] = bars.p[i & 1] + 16 * w;
      ptx::tmem_wait_ld();
      if (upper) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x = probability(fmaf(__uint_as_float(v[e]), c, kKeysHome ? -stat[e] : -own_lse));
          if (e < lo || e >= hi) x = 0.f;
          p[e][home] = x;
          v[e] = __float_as_uint(x);
        }
        named_barrier(1 + w, 128);
      } else {
        named_barrier(1 + w, 128);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = p[e][home] * (__uint_as_float(v[e]) - (kKeysHome ? stat[e] : own_delta));
          v[e] = e < lo || e >= hi ? 0u : __float_as_uint(x);
        }
      }
      // over S, which the group's upper rows have read (the lower rows' half of it is not used)
      if (sums) put_planes(v, slot + 16 * w, slot + kThird + 8 * w);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      arrive_warp(&bars.p_full[i & 1]);
      row += kStep;
      if (--left == 0) {                                // the next head's queries
        row = first + 16 * w;
        left = per;
      }
    };
    // the sums of step i, out of TMEM
    auto take = [&](int i) {
      if (ok) ok = wait_warp(&bars.sum_full, i & 1);
      ptx::tc_fence_after();
      if (sums) add_columns(total, total_at);
      ptx::tc_fence_before();
      arrive_warp(&bars.sum_free);
    };
    for (int i = 0; i < n; i += 2) {
      for (int j = i; j < i + 2 && j < n; ++j) pairs(j);
      for (int j = i; j < i + 2 && j < n; ++j) take(j);
    }
    if (!ok && lane == 0) report_timeout(status);
    if (sums && r < rows) {
      const Heads& t = kKeysHome ? (upper ? a.dv : a.dk) : a.dq;
      float* out = static_cast<float*>(t.p) + int64_t(b) * t.sb + int64_t(h) * t.sh + int64_t(r) * t.sl;
      const bool zero = n == 0 || (kKeysHome && r >= keys);
      const float by = !ok ? __uint_as_float(0x7FC00000u) : kKeysHome && upper ? 1.0f : a.scale;
#pragma unroll
      for (int cb = 0; cb < 64; cb += 32) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = zero ? 0u : __float_as_uint(total[cb + e]);
        if (64 * w + cb < a.dim) store_columns(out, 64 * w + cb, a.dim, v, by);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 10) ptx::tmem_dealloc(tmem, kTmemCols);
}

// The first `key_blocks` blocks own keys, the others queries.
__global__ void __launch_bounds__(kThreads, 1)
    attention_wide_backward_kernel(AttentionArgs a, unsigned* status, const __grid_constant__ Maps key_maps,
                                   const __grid_constant__ Maps query_maps, unsigned key_blocks) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ BackwardShared bars;
  if (blockIdx.x < key_blocks)
    wide_block<true>(a, status, key_maps.m, blockIdx.x, smem_raw, bars);
  else
    wide_block<false>(a, status, query_maps.m, blockIdx.x - key_blocks, smem_raw, bars);
}

constexpr int kForwardSmem = 1024 + 3 * kPlane128 + kStages * kTileBytes;
constexpr int kBackwardSmem = 1024 + 3 * kPlane128 + kStages * 2 * kStepBytes;

bool plane_map(const AttentionArgs& a, CUtensorMap* map, int which, int rows) {
  const bool keyed = which == 1 || which == 2;
  const int64_t length = keyed ? a.lk : a.lq, heads = keyed ? a.hkv : a.hq;
  return make_map(map, planes_of(a.planes[which], length, heads, 128), 3 * int64_t(a.batch), length, heads, 128, rows);
}

}  // namespace

cudaError_t launch_attention_wide_forward(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([](int) {
    return cudaFuncSetAttribute(attention_wide_forward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kForwardSmem);
  });
  unsigned* status = nullptr;
  if (e == cudaSuccess) e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  Maps maps{};
  if (!plane_map(a, &maps.m[0], 0, 128) || !plane_map(a, &maps.m[1], 1, kKeys) || !plane_map(a, &maps.m[2], 2, kKeys))
    return cudaErrorInvalidValue;
  const int64_t blocks = (int64_t(a.lq) + 127) / 128 * a.hq * a.batch;
  attention_wide_forward_kernel<<<static_cast<unsigned>(blocks), kThreads, kForwardSmem, stream>>>(a, status, maps);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_attention_wide_backward(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = once.run([](int) {
    return cudaFuncSetAttribute(attention_wide_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBackwardSmem);
  });
  unsigned* status = nullptr;
  if (e == cudaSuccess) e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  Maps key_maps{}, query_maps{};
  if (!plane_map(a, &key_maps.m[0], 1, kHome) || !plane_map(a, &key_maps.m[1], 2, kHome) ||
      !plane_map(a, &key_maps.m[2], 0, kStep) || !plane_map(a, &key_maps.m[3], 3, kStep) ||
      !plane_map(a, &query_maps.m[0], 0, kHome) || !plane_map(a, &query_maps.m[1], 3, kHome) ||
      !plane_map(a, &query_maps.m[2], 1, kStep) || !plane_map(a, &query_maps.m[3], 2, kStep))
    return cudaErrorInvalidValue;
  const int64_t key_blocks = a.dk.p ? (int64_t(a.lk) + kHome - 1) / kHome * a.hkv * a.batch : 0;
  const int64_t query_blocks = a.dq.p ? (int64_t(a.lq) + kHome - 1) / kHome * a.hq * a.batch : 0;
  if (key_blocks + query_blocks == 0) return cudaSuccess;
  attention_wide_backward_kernel<<<static_cast<unsigned>(key_blocks + query_blocks), kThreads, kBackwardSmem, stream>>>(
      a, status, key_maps, query_maps, static_cast<unsigned>(key_blocks));
  note_launch();
  return cudaGetLastError();
}

}  // namespace det
