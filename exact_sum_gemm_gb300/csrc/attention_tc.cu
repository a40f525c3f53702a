// Attention on the tensor cores (tcgen05), forward and backward.  The formulas,
// masks and the treatment of what masks hide are those of attention.cu; here
// the products run on bf16 operands with f32 accumulators in TMEM.
//
// bf16 (one plane): the probabilities are rounded to bf16 where they enter a
// product; the relative error 2^-9 of each is the operator's largest.
//
// f32 (three planes; head dimensions above 64: attention_wide.cu): an f32 value is the sum of
// three bf16 values, x = x0 + x1 + x2 + at most 2^-24 |x|, and a product of two
// such sums is taken as the six bf16 products x_i y_j with i + j <= 2, smallest
// first into the same accumulator; what is left out is below 2^-23 of |x y|.
// Q, K, V and dO are split once into planes in scratch (attention_split_kernel),
// P and dS as they are written to TMEM.  The tensor cores cut, not round, what
// does not fit when they add to an accumulator: sums kept in TMEM over all of
// 1024 keys were off by 8e-6.  So O and the gradients are taken out of TMEM
// after every step and summed in registers, where the cuts of a step's four or
// eight large products are all that is left.
//
// One block per SM, 12 warps:
//   warps 0-3, 4-7  two softmax groups, a thread per accumulator row
//   warp 8          TMA loads of 128-byte-swizzled tiles into a ring of stages
//                   (rows past the end and columns past the head dimension
//                   read as zero)
//   warp 9          goes over the tiles that need it before they are used: rows
//                   past a key length become zero, and under the causal
//                   diagonal non-finite values, which are reported
//   warps 10, 11    lane 0 issues the products that give S (and dP), and those
//                   that take P (and dS); warp 10 also allocates TMEM.  (One
//                   thread for both left the tensor cores idle for 40 % of a
//                   backward step: its waits and commits cost as much as the
//                   issue.)
// Tensors that a tensor map cannot describe (a base or stride off 16 bytes, a
// stride of 0) are loaded by warps 8 and 9 with 16-byte cp.async, or element by
// element (2 x 4096, 16/4 heads of 128, forward and backward: 852 us by cp.async
// where TMA took 669; its issue and its fences are the longest chain of a step).
//
// Forward: a block owns two tiles of 128 queries of a head, one per softmax
// group, and goes over the keys 64 at a time.  S = Q K^T lands in one of two
// TMEM slots of the half; the group takes the running maximum, writes P over S
// as bf16, and O += P V takes P from TMEM as its A operand, V as it lies in
// memory (MN-major).  The next S is computed meanwhile, so a group never waits
// for its own products.  O is rescaled only where
// a row's maximum has grown by more than 2^8 since its reference was taken; the
// decision is the row's own, so a row's bits do not depend on its neighbours.
//
// Backward: one launch, two kinds of block.  In the first a block owns 128 keys of
// a key head and goes over the queries of every head that shares it: S^T = K Q^T,
// dP^T = V dO^T, then dV += P^T dO and dK += dS^T Q, P^T and dS^T from TMEM.  In
// the second kind it owns 128 queries and goes over the keys: S = Q K^T, dP = dO
// V^T, dQ += dS K.  S and dP are computed twice (seven products instead of five),
// which is the price of sums without atomics and without f32 gradients in memory.
// The two softmax groups share a step's columns.
//   bf16: steps of 128 rows, as products 64 columns wide wait for shared memory to
// read their other operand (48 cycles in place of 32).  TMEM then holds one S
// and one dP beside dV and dK: P is written first, and while its product runs
// dS is taken from P in registers.  With dQ alone there is room for two S, so
// that the next one is ready when a step's softmax ends.  (64 rows and two
// slots of both took 482 us where this takes 434, 2 x 4096 causal with the
// statistics; 244 and 218, 2 x 2048, 16 heads of 128; but 15.1 and 16.5, 64 rows of
// 8 heads of 64, where half of a step is empty.)
//   Three planes: steps of 64 rows, two slots of S and dP, one with the softmax,
// the products of the other running.
//
// bf16, 2 x 4096 causal, 16/4 heads of 128: forward 142 us (968 TFLOP/s of the
// visible pairs' products), backward 392 us (877 counting five products, 1228
// counting the seven; a plain product reaches 1867).  Whole tiles along the
// diagonal come on top.  The tensor pipe is busy for 41 and 53 % of the cycles,
// the issue slots are for 49 and 33 %: neither is at its limit.  What is left of
// backward is the chain of a step (products, TMEM read, exponentials, TMEM write,
// products); forward's waits have not been measured, the start and end of a block
// are an eighth of its time.  f32 2 x 1024, 8 heads of 64: split 7, forward 33,
// split with statistics 8, backward 68 us, six times the products of bf16.
//
// Every wait is bounded (about 2 s); where one runs out the outputs are NaN and
// the library's device status records it.
#include "attention_tc.cuh"

namespace det {
namespace {

// ------------------------------------------------------------------ forward
constexpr int kFwdStages = 8;                           // K and V tiles in turn (three planes: 4)
constexpr int kKeys = 64;

struct FwdBars {
  uint64_t q_full, full[kFwdStages], empty[kFwdStages], cleaned[kFwdStages], s_full[2][2], p_full[2][2], o_done[2][2];
  uint64_t drained;
  uint32_t tmem;
  int bad;
};

// maps: Q, K, V.
template <int kPlanes, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_forward_kernel(AttentionArgs a, unsigned* status, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ FwdBars bars;
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  typedef typename std::conditional<kPlanes == 3, float, bf16>::type Out;
  constexpr int kStages = kPlanes == 3 ? kFwdStages / 2 : kFwdStages;
  const int panels = kPlanes == 1 && a.dim > 64 ? 2 : 1;
  const uint32_t half_bytes = panels * kPlanes * panel_bytes(128);
  const uint32_t tile_bytes = panels * kPlanes * panel_bytes(kKeys);
  const uint32_t ring = base + 2 * half_bytes;

  // block -> 256 (128) queries of a head, the longest rows of a causal mask first
  const int own = 128 * a.halves, tiles = (a.lq + own - 1) / own;
  const int64_t rest = blockIdx.x / a.hq;
  const int h = static_cast<int>(blockIdx.x - rest * a.hq), b = static_cast<int>(rest / tiles);
  const int tile = tiles - 1 - static_cast<int>(rest - int64_t(b) * tiles);
  const int hk = h / (a.hq / a.hkv), i0 = tile * own;
  const int keys = keys_of(a, b), offset = a.lk - a.lq;
  const int ksteps = (a.dim + 15) / 16;
  // key tiles of each half
  int n[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = i0 + 128 * t;
    int end = keys;
    if (a.causal) end = max(0, min(end, min(first + 128, a.lq) + offset));
    n[t] = first < a.lq && t < a.halves ? (end + kKeys - 1) / kKeys : 0;
  }
  const int n_all = max(n[0], n[1]);

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars.q_full, kTma ? 1 : kLoaders);
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&bars.full[s], kTma ? 1 : kLoaders);
      ptx::mbar_init(&bars.empty[s], kTma && kPlanes == 1 && (s & 1) ? 2 : 1);   // (V: and warp 9)
      ptx::mbar_init(&bars.cleaned[s], 32);
    }
    for (int t = 0; t < 2; ++t) {
      for (int u = 0; u < 2; ++u) {
        ptx::mbar_init(&bars.s_full[t][u], 1);
        ptx::mbar_init(&bars.p_full[t][u], 4);
        ptx::mbar_init(&bars.o_done[t][u], 1);
      }
    }
    ptx::mbar_init(&bars.drained, 1);
    bars.bad = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 10) {
    ptx::tmem_alloc(&bars.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // Two slots of S of each half, at 128 t + 64 u; O at 256 + 128 t (three planes: the third plane of
  // P at 256 + 64 t + 32 u, O at 384 + 64 t)
  const uint32_t tmem = bars.tmem;
  constexpr uint32_t kO = kPlanes == 3 ? 384 : 256, kOStep = kPlanes == 3 ? 64 : 128;

  // V of a key tile that the causal diagonal crosses for either half, or that holds rows past the
  // length (TMA reads zeros past the tensor's end only)
  auto crosses = [&](int j) { return a.causal && j * kKeys + kKeys - 1 > i0 + offset; };
  auto special = [&](int j) {
    return kPlanes == 1 && (crosses(j) || (keys < a.lk && (j + 1) * kKeys > keys));   // (planes are clean)
  };

  if (kTma && warp == 8) {
    if (lane == 0 && n_all > 0) {
      ptx::mbar_arrive_expect_tx(&bars.q_full, a.halves * half_bytes);
      tma_rows<kPlanes, 128>(base, &maps.m[0], &bars.q_full, panels, i0, h, b, a.batch);
      if (a.halves == 2)
        tma_rows<kPlanes, 128>(base + half_bytes, &maps.m[0], &bars.q_full, panels, i0 + 128, h, b, a.batch);
      bool ok = true;
      int it = 0;                                       // K and V of every key tile in turn
      for (; it < 2 * n_all; ++it) {
        const int s = it % kStages;
        if (!wait_bounded(&bars.empty[s], ((it / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        ptx::mbar_arrive_expect_tx(&bars.full[s], tile_bytes);
        tma_rows<kPlanes, kKeys>(ring + s * tile_bytes, &maps.m[1 + (it & 1)], &bars.full[s], panels, it / 2 * kKeys,
                                 hk, b, a.batch);
      }
      // nothing in flight at the block's end, however it comes
      if (!wait_bounded(&bars.q_full, 0)) ok = false;
      for (int j = max(0, it - kStages); j < it; ++j)
        if (!wait_bounded(&bars.full[j % kStages], (j / kStages) & 1)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (kTma && kPlanes == 1 && warp == 9) {
    const Source v = source(a.v, b, hk, keys, a.dim);
    for (int j = 0; j < n_all; ++j) {
      // (every V in turn, none given back before: a wait tells a phase from the one before it, not
      // from older ones)
      const int item = 2 * j + 1, s = item % kStages;
      if (!wait_warp(&bars.full[s], (item / kStages) & 1)) {
        if (lane == 0) report_timeout(status);
        break;
      }
      if (special(j)) {
        bool found = false;
        for (int tid = lane; tid < kLoaders; tid += 32)
          found |= clean_rows<kKeys>(ring + s * tile_bytes, v, j * kKeys, keys == a.lk, crosses(j), tid);
        if (found) bars.bad = 1;
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars.cleaned[s]);
      }
      arrive_warp(&bars.empty[s]);
    }
  } else if (!kTma && (warp == 8 || warp == 9)) {
    const int tid = threadIdx.x - 256;
    const Source q = source(a.q, b, h, a.lq, a.dim);
    const Source k = source(a.k, b, hk, keys, a.dim), v = source(a.v, b, hk, keys, a.dim);
    bool ok = true;
    // item 0: the queries; then K and V of every key tile in turn
    const int items = n_all > 0 ? 1 + 2 * n_all : 0;
    int it = 0, fin = 0;                                // the items to start and to finish next
    auto finish = [&]() {
      const int it = fin++;
      if (it == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars.q_full);
        return;
      }
      const int s = (it - 1) % kStages, j = (it - 1) / 2;
      if (((it - 1) & 1) && crosses(j) && clean_rows<kKeys>(ring + s * tile_bytes, v, j * kKeys, true, true, tid))
        bars.bad = 1;
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&bars.full[s]);
    };
    // A full ring is the time to hand over what has arrived.
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (phase_over(bar, parity)) return true;
      cp_async_wait<0>();
      while (fin < it) finish();
      return wait_bounded(bar, parity);
    };
    for (; it < items && ok; ++it) {
      if (it == 0) {
        load_rows<128>(base, q, i0, tid);
        if (a.halves == 2) load_rows<128>(base + half_bytes, q, i0 + 128, tid);
      } else {
        const int s = (it - 1) % kStages;
        if (!acquire(&bars.empty[s], (((it - 1) / kStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        load_rows<kKeys>(ring + s * tile_bytes, ((it - 1) & 1) ? v : k, (it - 1) / 2 * kKeys, tid);
      }
      cp_async_commit();
      if (it >= fin + kAhead) {
        cp_async_wait<kAhead>();
        finish();
      }
    }
    cp_async_wait<0>();
    while (ok && fin < it) finish();
    if (!ok && tid == 0) report_timeout(status);
  } else if (warp == 10) {
    if (lane == 0 && n_all > 0) {
      const uint32_t idesc_s = ptx::idesc_bf16_f32(128, kKeys);
      bool ok = wait_bounded(&bars.q_full, 0);
      for (int j = 0; j < n_all && ok; ++j) {
        const int item = 2 * j, s = item % kStages;
        ok = wait_bounded(&bars.full[s], (item / kStages) & 1);
        for (int t = 0; t < 2 && ok; ++t) {
          if (j >= n[t]) continue;
          // (P of the step before the last is where S goes)
          if (j >= 2 && !wait_bounded(&bars.o_done[t][j & 1], ((j >> 1) - 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          product_ss<kPlanes, 128, kKeys, kPlanes == 3 ? 1 : 2>(tmem + 128 * t + 64 * (j & 1), base + t * half_bytes,
                                          ring + s * tile_bytes, ksteps, idesc_s);
          ptx::mma_commit(&bars.s_full[t][j & 1]);
        }
        // (only where the loaders wait for it: nothing arrives after the block's end)
        if (item + kStages < 2 * n_all) ptx::mma_commit(&bars.empty[s]);
      }
      if (!ok) report_timeout(status);
    }
  } else if (warp == 11) {
    if (lane == 0 && n_all > 0) {
      const uint32_t idesc_o = ptx::idesc_bf16_f32(128, ksteps * 16) | kMnB;
      uint32_t clean_phase = 0;                         // a bit per stage
      bool ok = true;
      for (int j = 0; j < n_all && ok; ++j) {
        const int item = 2 * j + 1, s = item % kStages;
        ok = wait_bounded(&bars.full[s], (item / kStages) & 1);
        if (kTma && ok && special(j)) {
          ok = wait_bounded(&bars.cleaned[s], clean_phase >> s & 1u);
          clean_phase ^= 1u << s;
        }
        for (int t = 0; t < 2 && ok; ++t) {
          if (j >= n[t]) continue;
          if (!wait_bounded(&bars.p_full[t][j & 1], (j >> 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          product_ts<kPlanes, kKeys, 16, kPlanes == 3 ? 1 : 2>(tmem + kO + kOStep * t, tmem + 128 * t + 64 * (j & 1),
                                         tmem + 256 + 64 * t + 32 * (j & 1), ring + s * tile_bytes, idesc_o,
                                         kPlanes == 1 && j > 0);
          ptx::mma_commit(&bars.o_done[t][j & 1]);
        }
        if (item + kStages < 2 * n_all) ptx::mma_commit(&bars.empty[s]);
      }
      // (S before them is done too: P waited for it)
      ptx::mma_commit(&bars.drained);
      if (!wait_bounded(&bars.drained, 0)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp < 8) {
    const int t = warp >> 2, row = 32 * (warp & 3) + lane, i = i0 + 128 * t + row;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_at = tmem + lanes + kO + kOStep * t;
    const float c = a.scale * kLog2e;
    const int last = a.causal ? min(keys, i + offset + 1) : keys;   // keys [0, last) are visible
    float ref = -INFINITY, l = 0.f;
    float o_sum[kPlanes == 3 ? kNarrowDim : 1];         // three planes: O so far
#pragma unroll
    for (float& x : o_sum) x = 0.f;
    bool ok = true;
    for (int j = 0; j < n[t]; ++j) {
      if (!wait_warp(&bars.s_full[t][j & 1], (j >> 1) & 1)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const uint32_t s_at = tmem + lanes + 128 * t + 64 * (j & 1);
      const int seen = last - j * kKeys;                // columns [0, seen) are visible
      const bool whole = __all_sync(0xFFFFFFFFu, seen >= kKeys);
      uint32_t v[kKeys / 32][32];
#pragma unroll
      for (int cb = 0; cb < kKeys / 32; ++cb) ptx::tmem_ld32(s_at + 32 * cb, v[cb]);
      ptx::tmem_wait_ld();
      if (!whole) {
#pragma unroll
        for (int cb = 0; cb < kKeys / 32; ++cb) hide(v[cb], seen - 32 * cb, c);
      }
      float top = c < 0.f ? row_extreme<true>(v) : row_extreme<false>(v);
      top = c == 0.f ? (seen > 0 ? top * c : -INFINITY) : top * c;
      const bool grow = top > ref + 8.0f || (ref == -INFINITY && top != -INFINITY);
      const bool any_grow = __any_sync(0xFFFFFFFFu, grow);
      float by = 1.0f;
      if (any_grow) {
        const float next = grow ? top : ref;
        if (grow) by = exp2_approx(ref - next);
        if (kPlanes == 1 && j > 0) {
          if (!wait_warp(&bars.o_done[t][(j - 1) & 1], ((j - 1) >> 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          for (int cb = 0; cb < ksteps * 16; cb += 32) {
            uint32_t x[32];
            ptx::tmem_ld32(o_at + cb, x);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * by);
            ptx::tmem_st32(o_at + cb, x);
          }
        }
        l *= by;
        ref = next;
      }
      const float sub = ref == -INFINITY ? 0.f : ref;
      float by_c = c;
      if (__any_sync(0xFFFFFFFFu, fabsf(sub) >= kFar)) {
#pragma unroll
        for (int cb = 0; cb < kKeys / 32; ++cb) scale_far(v[cb], sub, c);
        if (fabsf(sub) >= kFar) by_c = 1.f;
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int cb = 0; cb < kKeys / 32; ++cb) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float p = exp2_approx(fmaf(__uint_as_float(v[cb][e]), by_c, -sub));
          if (c == 0.f && !whole && 32 * cb + e >= seen) p = 0.f;       // (0 x inf)
          sum[e & 3] += p;
          v[cb][e] = __float_as_uint(p);
        }
        // P over S, which is in registers
        if constexpr (kPlanes == 1) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            uint32_t part[1];
            split_pair<1>(__uint_as_float(v[cb][2 * e]), __uint_as_float(v[cb][2 * e + 1]), part);
            w[e] = part[0];
          }
          tmem_st16(s_at + 16 * cb, w);
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = v[cb][16 * g + e];
            put_planes(x, s_at + 32 * cb + 16 * g, tmem + lanes + 256 + 64 * t + 32 * (j & 1) + 16 * cb + 8 * g);
          }
        }
      }
      if constexpr (kPlanes == 3) {
        // the product of the step before has run beside this: O of it, taken with its reference,
        // joins the sum before the next product writes there
        if (j > 0) {
          if (!wait_warp(&bars.o_done[t][(j - 1) & 1], ((j - 1) >> 1) & 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          add_columns(o_sum, o_at);
        }
        if (any_grow) {
#pragma unroll
          for (int e = 0; e < kNarrowDim; ++e) o_sum[e] *= by;
        }
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      arrive_warp(&bars.p_full[t][j & 1]);
    }
    if (ok && n[t] > 0) {
      ok = wait_warp(&bars.o_done[t][(n[t] - 1) & 1], ((n[t] - 1) >> 1) & 1);
      ptx::tc_fence_after();
      if constexpr (kPlanes == 3) add_columns(o_sum, o_at);
    }
    if (!ok && lane == 0) report_timeout(status);
    const float inv = !ok ? __uint_as_float(0x7FC00000u) : l == 0.f ? 0.f : 1.0f / l;
    Out* o = static_cast<Out*>(a.o.p) + int64_t(b) * a.o.sb + int64_t(h) * a.o.sh + int64_t(i) * a.o.sl;
    for (int cb = 0; cb < ksteps * 16; cb += 32) {
      uint32_t v[32];
      if (kPlanes == 3) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = __float_as_uint(cb == 0 ? o_sum[kPlanes == 3 ? e : 0] : o_sum[kPlanes == 3 ? 32 + e : 0]);
      } else if (n[t] > 0) {
        ptx::tmem_ld32(o_at + cb, v);
        ptx::tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
      }
      if (i < a.lq && t < a.halves) store_columns(o, cb, a.dim, v, inv);
    }
    if (i < a.lq && t < a.halves)
      a.lse[(int64_t(b) * a.hq + h) * a.lq + i] =
          !ok ? inv : l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (kPlanes == 1 && a.flags && threadIdx.x == 0) a.flags[(int64_t(b) * tiles + tile) * a.hq + h] = bars.bad;
  if (warp == 10) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------ backward
constexpr int kBwdStages = 4;                           // (three planes: 2)
constexpr int stages_of(int planes) { return planes == 3 ? 2 : kBwdStages; }
constexpr int kStep = 64;
// Whether the steps are of 128 rows: then with four tiles, two of Q and two of dO, or three of K and
// one of V, which is used by the first product alone (with one of dO as well: 436 -> 468 us).
constexpr bool long_steps(int planes) { return planes == 1; }

struct BwdBars {
  alignas(16) float lse[kBwdStages * kStep], delta[kBwdStages * kStep];
  uint64_t home_full, full[kBwdStages], empty[kBwdStages], cleaned[kBwdStages], s_full[2], p_full[2], slot_free[2], acc_full;
  uint64_t sum_full, sum_free;                          // three planes: a step's sums
  // long steps: dP is there, in registers; the second operand's place
  uint64_t dp_full, dp_free, v_full[2], v_empty[2];
  uint32_t tmem;
  int bad;
};

// Block `block` of the keys' (kKeysHome: it owns 128 keys, dk and dv) or of the
// queries' (128 queries, dq).  maps: the home tiles' tensors (K, V or Q, dO),
// the steps' (Q, dO or K, V).
template <int kPlanes, bool kKeysHome, bool kTma>
__device__ __forceinline__ void backward_block(const AttentionArgs& a, unsigned* status, const CUtensorMap* maps,
                                               int64_t block, unsigned char* smem_raw, BwdBars& bars) {
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  typedef typename std::conditional<kPlanes == 3, float, bf16>::type Out;
  constexpr bool kLong = long_steps(kPlanes);
  constexpr int kStages = !kLong ? stages_of(kPlanes) : kKeysHome ? 2 : 3, kSeconds = kKeysHome ? 2 : 1;
  constexpr int kRows = kLong ? 2 * kStep : kStep;
  const int panels = kPlanes == 1 && a.dim > 64 ? 2 : 1;
  const uint32_t home_bytes = panels * kPlanes * panel_bytes(128);
  const uint32_t step_bytes = panels * kPlanes * panel_bytes(kRows);
  // stages of two step tiles; long steps: of Q or K alone, then kSeconds places for dO or V, which
  // are done with a product earlier
  const uint32_t ring = base + 2 * home_bytes, stage_bytes = (kLong ? 1 : 2) * step_bytes;
  auto second = [&](int i) { return ring + (kLong ? kStages + i % kSeconds : 2 * (i % kStages) + 1) * step_bytes; };

  const int rows = kKeysHome ? a.lk : a.lq, heads = kKeysHome ? a.hkv : a.hq;
  const int tiles = (rows + 127) / 128;
  const int64_t rest = block / heads;
  const int h = static_cast<int>(block - rest * heads), b = static_cast<int>(rest / tiles);
  int tile = static_cast<int>(rest - int64_t(b) * tiles);
  if (!kKeysHome) tile = tiles - 1 - tile;              // most work first under a causal mask
  const int r0 = tile * 128, share = a.hq / a.hkv;
  const int keys = keys_of(a, b), offset = a.lk - a.lq;
  const int ksteps = (a.dim + 15) / 16;
  // the steps: `per` tiles of kRows rows from `first`, for each of `streams` heads
  int first = 0, end = kKeysHome ? a.lq : keys;
  if (a.causal) {
    if (kKeysHome) first = max(0, r0 - offset) / kRows * kRows;
    else end = max(0, min(end, min(r0 + 128, a.lq) + offset));
  }
  int per = end > first ? (end - first + kRows - 1) / kRows : 0;
  if (kKeysHome && r0 >= keys) per = 0;
  const int n = per * (kKeysHome ? share : 1);
  const int h_first = kKeysHome ? h * share : h / share;

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars.home_full, kTma ? 1 : kLoaders);
    for (int s = 0; s < kBwdStages; ++s) {
      ptx::mbar_init(&bars.full[s], kTma ? 1 : kLoaders);
      ptx::mbar_init(&bars.empty[s], kTma && kPlanes == 1 ? 2 : 1);   // (and warp 9)
      ptx::mbar_init(&bars.cleaned[s], 32);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&bars.s_full[t], 1);
      ptx::mbar_init(&bars.p_full[t], 8);
      ptx::mbar_init(&bars.slot_free[t], 1);
    }
    ptx::mbar_init(&bars.acc_full, 1);
    ptx::mbar_init(&bars.sum_full, 1);
    ptx::mbar_init(&bars.sum_free, 8);
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(&bars.v_full[t], kTma ? 1 : kLoaders);
      ptx::mbar_init(&bars.v_empty[t], kTma && kKeysHome ? 2 : 1);
    }
    ptx::mbar_init(&bars.dp_full, 1);
    ptx::mbar_init(&bars.dp_free, 8);
    bars.bad = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 10) {
    ptx::tmem_alloc(&bars.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // bf16: S (128 columns), which P overwrites, dP (128), which dS overwrites, dv, dk; or two slots of
  // S, which dS overwrites, dP, dq.  Three planes: two slots of S (64) and dP (64), which P and dS
  // overwrite, each with 32 columns more for the third; then dv, then dk or dq.
  const uint32_t tmem = bars.tmem;
  constexpr uint32_t kDp = !kLong ? 96 : kKeysHome ? 128 : 256, kSlot = !kLong ? 2 * kDp : kKeysHome ? 0 : 128;
  constexpr uint32_t kDv = kLong ? 256 : 2 * kSlot, kAcc = kLong ? 384 : 448;

  // a step's tile that the diagonal crosses, or that holds rows past the key length
  auto crosses = [&](int row) {
    return a.causal && (kKeysHome ? r0 + 127 > row + offset : row + kRows - 1 > r0 + offset);
  };
  auto special = [&](int row) {                         // (planes are clean)
    return kPlanes == 1 && (crosses(row) || (!kKeysHome && keys < a.lk && row + kRows > keys));
  };
  auto step_sources = [&](int head, Source& x, Source& y) {
    if (kKeysHome) {
      x = source(a.q, b, head, a.lq, a.dim);
      y = source(a.dout, b, head, a.lq, a.dim);
    } else {
      x = source(a.k, b, head, keys, a.dim);
      y = source(a.v, b, head, keys, a.dim);
    }
  };

  if (kTma && warp == 8) {
    if (lane == 0 && n > 0) {
      ptx::mbar_arrive_expect_tx(&bars.home_full, 2 * home_bytes);
      tma_rows<kPlanes, 128>(base, &maps[0], &bars.home_full, panels, r0, h, b, a.batch);
      tma_rows<kPlanes, 128>(base + home_bytes, &maps[1], &bars.home_full, panels, r0, h, b, a.batch);
      bool ok = true;
      int i = 0, seconds = 0, head = h_first, row = first;
      // long steps: the second tile, in a place of its own
      auto load_second = [&]() {
        if (!kLong) return true;
        uint64_t* full = &bars.v_full[i % kSeconds];
        if (!wait_bounded(&bars.v_empty[i % kSeconds], ((i / kSeconds) & 1) ^ 1)) return false;
        ptx::mbar_arrive_expect_tx(full, step_bytes);
        tma_rows<kPlanes, kRows>(second(i), &maps[3], full, panels, row, head, b, a.batch);
        ++seconds;
        return true;
      };
      while (i < n) {
        const int s = i % kStages;
        if (kKeysHome) ok = load_second();              // (dO: free before Q)
        if (ok) ok = wait_bounded(&bars.empty[s], ((i / kStages) & 1) ^ 1);
        if (!ok) break;
        ptx::mbar_arrive_expect_tx(&bars.full[s], stage_bytes + (kKeysHome ? 2 * kRows * 4 : 0));
        tma_rows<kPlanes, kRows>(ring + s * stage_bytes, &maps[2], &bars.full[s], panels, row, head, b, a.batch);
        if (!kLong) tma_rows<kPlanes, kRows>(second(i), &maps[3], &bars.full[s], panels, row, head, b, a.batch);
        if (kKeysHome) {
          const int64_t q = (int64_t(b) * a.hq + head) * a.stat_stride + row;
          bulk_load(bars.lse + s * kRows, a.lse2 + q, kRows * 4, &bars.full[s]);
          bulk_load(bars.delta + s * kRows, a.delta + q, kRows * 4, &bars.full[s]);
        }
        if (!kKeysHome) ok = load_second();
        ++i;
        if (!ok) break;
        row += kRows;
        if (row >= end) {
          row = first;
          ++head;
        }
      }
      // nothing in flight at the block's end, however it comes
      if (!wait_bounded(&bars.home_full, 0)) ok = false;
      for (int j = max(0, i - kStages); j < i; ++j)
        if (!wait_bounded(&bars.full[j % kStages], (j / kStages) & 1)) ok = false;
      for (int j = max(0, seconds - kSeconds); j < seconds; ++j)
        if (!wait_bounded(&bars.v_full[j % kSeconds], (j / kSeconds) & 1)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (kTma && kPlanes == 1 && warp == 9) {
    Source x, y;
    step_sources(h_first, x, y);                        // (the shape is every head's)
    int row = first;
    for (int i = 0; i < n; ++i) {
      // (every step in turn, no tile given back before: a wait tells a phase from the one before it,
      // not from older ones)
      const int s = i % kStages;
      if (!wait_warp(&bars.full[s], (i / kStages) & 1) || 
          (kKeysHome && !wait_warp(&bars.v_full[i % kSeconds], (i / kSeconds) & 1))) {
        if (lane == 0) report_timeout(status);
        break;
      }
      if (special(row)) {
        const uint32_t at = ring + s * stage_bytes;
        bool found = false;
        for (int tid = lane; tid < kLoaders; tid += 32) {
          found |= clean_rows<kRows>(at, x, row, kKeysHome || keys == a.lk, crosses(row), tid);
          if (kKeysHome) found |= clean_rows<kRows>(second(i), y, row, true, true, tid);
        }
        if (found) bars.bad = 1;
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars.cleaned[s]);
      }
      arrive_warp(&bars.empty[s]);
      if (kKeysHome) arrive_warp(&bars.v_empty[i % kSeconds]);
      row = row + kRows < end ? row + kRows : first;
    }
  } else if (!kTma && (warp == 8 || warp == 9)) {
    const int tid = threadIdx.x - 256;
    bool ok = true;
    int it = 0, fin = 0, fin_row = first;               // the items to start and to finish next
    // item 0: the home tiles; item 1 + i: step i
    Source x, y;
    step_sources(h_first, x, y);
    auto finish = [&]() {
      const int it = fin++;
      if (it == 0) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&bars.home_full);
        return;
      }
      const int s = (it - 1) % kStages;
      const uint32_t at = ring + s * stage_bytes;
      if (crosses(fin_row)) {                           // what enters a sum over its rows
        bool found = clean_rows<kRows>(at, x, fin_row, true, true, tid);
        if (kKeysHome) found |= clean_rows<kRows>(second(it - 1), y, fin_row, true, true, tid);
        if (found) bars.bad = 1;
      }
      fin_row = fin_row + kRows < end ? fin_row + kRows : first;
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&bars.full[s]);
      if (kLong) ptx::mbar_arrive(&bars.v_full[(it - 1) % kSeconds]);
    };
    const int items = n > 0 ? 1 + n : 0;
    int head = h_first, row = first;
    auto acquire = [&](uint64_t* bar, uint32_t parity) {
      if (phase_over(bar, parity)) return true;
      cp_async_wait<0>();
      while (fin < it) finish();
      return wait_bounded(bar, parity);
    };
    for (; it < items; ++it) {
      if (it == 0) {
        Source u, w;
        if (kKeysHome) {
          u = source(a.k, b, h, keys, a.dim);
          w = source(a.v, b, h, keys, a.dim);
        } else {
          u = source(a.q, b, h, a.lq, a.dim);
          w = source(a.dout, b, h, a.lq, a.dim);
        }
        load_rows<128>(base, u, r0, tid);
        load_rows<128>(base + home_bytes, w, r0, tid);
      } else {
        const int s = (it - 1) % kStages;
        if (!acquire(&bars.empty[s], (((it - 1) / kStages) & 1) ^ 1) ||
            (kLong && !acquire(&bars.v_empty[(it - 1) % kSeconds], (((it - 1) / kSeconds) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const uint32_t at = ring + s * stage_bytes;
        load_rows<kRows>(at, x, row, tid);
        load_rows<kRows>(second(it - 1), y, row, tid);
        constexpr int kFours = kRows / 4;               // of lse, and of delta
        if (kKeysHome && tid < 2 * kFours) {
          const int64_t q = (int64_t(b) * a.hq + head) * a.stat_stride + row;
          const float* from = (tid < kFours ? a.lse2 : a.delta) + q + (tid % kFours) * 4;
          float* to = (tid < kFours ? bars.lse : bars.delta) + s * kRows + (tid % kFours) * 4;
          cp_async16(ptx::smem_addr(to), from, true);
        }
        row += kRows;
        if (row >= end) {
          row = first;
          ++head;
          if (it + 1 < items) step_sources(head, x, y);
        }
      }
      cp_async_commit();
      if (it >= fin + kAhead) {
        cp_async_wait<kAhead>();
        finish();
      }
    }
    cp_async_wait<0>();
    while (ok && fin < it) finish();
    if (!ok && tid == 0) report_timeout(status);
  } else if (warp == 10) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc_s = ptx::idesc_bf16_f32(128, kRows);
      bool ok = wait_bounded(&bars.home_full, 0);
      uint32_t clean_phase = 0;                         // a bit per stage
      int row = first;
      for (int i = 0; i < n && ok; ++i) {               // S and dP of step i into its slot
        const int s = i % kStages;
        ok = wait_bounded(&bars.full[s], (i / kStages) & 1);
        if (kTma && ok && special(row)) {
          ok = wait_bounded(&bars.cleaned[s], clean_phase >> s & 1u);
          clean_phase ^= 1u << s;
        }
        row = row + kRows < end ? row + kRows : first;
        // what lies where they go has been used: by the last step but one, or by the last
        if (kLong && kKeysHome) {
          if (ok && i >= 1) ok = wait_bounded(&bars.slot_free[0], (i - 1) & 1);
        } else if (ok && i >= 2) {
          ok = wait_bounded(&bars.slot_free[i & 1], ((i >> 1) - 1) & 1);
        }
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t at = ring + s * stage_bytes, d = tmem + kSlot * (i & 1);
        product_ss<kPlanes, 128, kRows, kPlanes == 3 ? 1 : 2>(d, base, at, ksteps, idesc_s);
        if constexpr (kLong) {
          ptx::mma_commit(&bars.s_full[kKeysHome ? 0 : i & 1]);
          if (kLong) ok = wait_bounded(&bars.v_full[i % kSeconds], (i / kSeconds) & 1);
          // (dP of the step before is in registers, or dS has been used)
          if (i > 0 && ok) ok = wait_bounded(kKeysHome ? &bars.slot_free[1] : &bars.dp_free, (i - 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
        }
        product_ss<kPlanes, 128, kRows, kPlanes == 3 ? 1 : 2>(kLong ? tmem + kDp : d + kDp, base + home_bytes,
                                                              second(i), ksteps, idesc_s);
        ptx::mma_commit(kLong ? &bars.dp_full : &bars.s_full[i & 1]);
        if (kLong && !kKeysHome && i + kSeconds < n) ptx::mma_commit(&bars.v_empty[i % kSeconds]);
      }
      if (!ok) report_timeout(status);
    }
  } else if (warp == 11) {
    if (lane == 0 && n > 0) {
      const uint32_t idesc_acc = ptx::idesc_bf16_f32(128, ksteps * 16) | kMnB;
      bool ok = true;
      // bf16: acc += A B over a step's 128 rows, of which A has the first 64 in 32 words at `from`, the
      // others 64 words on
      auto add_step = [&](uint32_t acc, uint32_t from, uint32_t b, bool add) {
        const uint64_t bd = desc_mn(b, panel_bytes(kRows));
#pragma unroll
        for (int k = 0; k < kRows / 16; ++k)
          mma_ts(acc, from + (k >> 2) * 64 + (k & 3) * 8, bd + k * (2048 >> 4), idesc_acc, add || k > 0);
      };
      for (int i = 0; i < n && ok; ++i) {               // the sums, once P and dS of step i are there
        const int s = i % kStages;
        const uint32_t at = ring + s * stage_bytes;
        if constexpr (kLong && kKeysHome) {
          ok = wait_bounded(&bars.p_full[0], i & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          add_step(tmem + kDv, tmem, second(i), i > 0);
          if (i + 1 < n) ptx::mma_commit(&bars.slot_free[0]);
          if (i + kSeconds < n) ptx::mma_commit(&bars.v_empty[i % kSeconds]);
          ok = wait_bounded(&bars.p_full[1], i & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          add_step(tmem + kAcc, tmem + kDp, at, i > 0);
          if (i + 1 < n) ptx::mma_commit(&bars.slot_free[1]);
          if (i + kStages < n) ptx::mma_commit(&bars.empty[s]);
          continue;
        }
        ok = wait_bounded(&bars.p_full[i & 1], (i >> 1) & 1);
        if (kPlanes == 3 && i > 0 && ok) ok = wait_bounded(&bars.sum_free, (i - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t p = tmem + kSlot * (i & 1);
        if constexpr (kLong) {
          add_step(tmem + kAcc, p, at, i > 0);
        } else {
          const uint32_t ds = p + kDp;
          if (kKeysHome) product_ts<kPlanes, kRows, 32, 1>(tmem + kDv, p, p + 64, at + step_bytes, idesc_acc, false);
          product_ts<kPlanes, kRows, 32, 1>(tmem + kAcc, ds, ds + 64, at, idesc_acc, false);
        }
        // (only where they are waited for: nothing arrives after the block's end)
        if (i + kStages < n) ptx::mma_commit(&bars.empty[s]);
        if (i + 2 < n) ptx::mma_commit(&bars.slot_free[i & 1]);
        if (kPlanes == 3) ptx::mma_commit(&bars.sum_full);
      }
      ptx::mma_commit(&bars.acc_full);                  // all of the above, and S and dP before them
      if (!wait_bounded(&bars.acc_full, 0)) ok = false;
      if (!ok) report_timeout(status);
    }
  } else if (warp < 8) {
    const int w = warp >> 2, r = r0 + 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    constexpr int kCols = kRows / 2;                    // the group's columns of a slot
    const uint32_t at = tmem + lanes + kCols * w;
    const float c = a.scale * kLog2e;
    float own_lse = INFINITY, own_delta = 0.f;          // of the thread's query
    if (!kKeysHome && r < a.lq) {
      const int64_t i = (int64_t(b) * a.hq + h) * a.stat_stride + r;
      own_lse = __ldg(a.lse2 + i);
      own_delta = __ldg(a.delta + i);
    }
    bool ok = true;
    int row = first + kCols * w, left = per;            // the group's first row of the step
    // three planes: the block's sums so far, dv of the first group and dk of the second, or half of dq
    float total[kPlanes == 1 ? 1 : kKeysHome ? kNarrowDim : kNarrowDim / 2];
#pragma unroll
    for (float& x : total) x = 0.f;
    const uint32_t total_at = tmem + lanes + (kKeysHome ? (w == 0 ? kDv : kAcc) : kAcc + 32 * w);
    // P and dS of step i
    auto pairs = [&](int i) {
      const uint32_t slot = kSlot * (i & 1);
      // (the second wait is over at once: it orders the loaders' lse and delta before their use)
      constexpr bool kOneSlot = kLong && kKeysHome;
      if (!wait_warp(&bars.s_full[kOneSlot ? 0 : i & 1], (kOneSlot ? i : i >> 1) & 1) ||
          (kKeysHome && !wait_warp(&bars.full[i % kStages], (i / kStages) & 1)))
        return false;
      ptx::tc_fence_after();
      // columns [lo, hi) of the group's are visible to the thread's row
      int lo = 0, hi = kCols;
      if (kKeysHome) {
        hi = a.lq - row;
        if (a.causal) lo = r - offset - row;
      } else {
        hi = keys - row;
        if (a.causal) hi = min(hi, r + offset + 1 - row);
      }
      const bool whole = __all_sync(0xFFFFFFFFu, lo <= 0 && hi >= kCols);
      const float* lse = bars.lse + i % kStages * kRows + kCols * w;
      const float* delta = bars.delta + i % kStages * kRows + kCols * w;
      // three planes: P and dS of 16 columns from column c0 of the 32, in place
      auto pair_columns = [&](uint32_t (&sv)[16], uint32_t (&dv)[16], int c0) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          float l[4] = {own_lse, own_lse, own_lse, own_lse};
          float d[4] = {own_delta, own_delta, own_delta, own_delta};
          if (kKeysHome) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse + c0 + e);
            const float4 d4 = *reinterpret_cast<const float4*>(delta + c0 + e);
            l[0] = l4.x, l[1] = l4.y, l[2] = l4.z, l[3] = l4.w;
            d[0] = d4.x, d[1] = d4.y, d[2] = d4.z, d[3] = d4.w;
          }
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            const float p = probability(fmaf(__uint_as_float(sv[e + f]), c, -l[f]));
            dv[e + f] = __float_as_uint(p * (__uint_as_float(dv[e + f]) - d[f]));
            sv[e + f] = __float_as_uint(p);
          }
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (c0 + e < lo || c0 + e >= hi) sv[e] = dv[e] = 0u;
        }
      };
      // zeroes for what the row does not see of 32 columns from c0 (apart, so that the rest has no
      // branches)
      auto hide = [&](uint32_t (&x)[32], int c0) {
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c0 + e < lo || c0 + e >= hi) x[e] = 0u;
        }
      };
      auto put_pairs = [&](const uint32_t (&x)[32], uint32_t to) {
        uint32_t word[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          uint32_t part[1];
          split_pair<1>(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]), part);
          word[e] = part[0];
        }
        tmem_st16(to, word);
      };
      // over the group's own columns, which are in registers
      if constexpr (kOneSlot) {
        // P of all 64 columns, for dv; dS from it when dP is there, while the products with P run
        uint32_t p[2][32];
        ptx::tmem_ld32(at, p[0]);
        ptx::tmem_ld32(at + 32, p[1]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse + 32 * h + e);
            const float by[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int f = 0; f < 4; ++f)
              p[h][e + f] = __float_as_uint(probability(fmaf(__uint_as_float(p[h][e + f]), c, -by[f])));
          }
          hide(p[h], 32 * h);
          put_pairs(p[h], at + 16 * h);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        arrive_warp(&bars.p_full[0]);
        if (!wait_warp(&bars.dp_full, i & 1)) return false;
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t dv[32];
          ptx::tmem_ld32(at + kDp + 32 * h, dv);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(delta + 32 * h + e);
            const float by[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int f = 0; f < 4; ++f)
              dv[e + f] = __float_as_uint(__uint_as_float(p[h][e + f]) * (__uint_as_float(dv[e + f]) - by[f]));
          }
          hide(dv, 32 * h);
          put_pairs(dv, at + kDp + 16 * h);
        }
      } else if constexpr (kLong) {
        // 32 columns at a time: P while dP is on its way, dS over the columns of S before them
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t sv[32], dv[32];
          ptx::tmem_ld32(at + slot + c0, sv);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            sv[e] = __float_as_uint(probability(fmaf(__uint_as_float(sv[e]), c, -own_lse)));
          if (c0 == 0) {
            if (!wait_warp(&bars.dp_full, i & 1)) return false;
            ptx::tc_fence_after();
          }
          ptx::tmem_ld32(at + kDp + c0, dv);
          ptx::tmem_wait_ld();
          if (c0 + 32 == kCols) {
            ptx::tc_fence_before();
            arrive_warp(&bars.dp_free);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            dv[e] = __float_as_uint(__uint_as_float(sv[e]) * (__uint_as_float(dv[e]) - own_delta));
          hide(dv, c0);
          put_pairs(dv, at + slot + c0 / 2);
        }
      } else {
#pragma unroll
        for (int c0 = 0; c0 < 32; c0 += 16) {
          uint32_t sv[16], dv[16];
          const uint32_t to = at + slot + c0, third = tmem + lanes + slot + 64 + 16 * w + c0 / 2;
          tmem_ld16(to, sv);
          tmem_ld16(to + kDp, dv);
          ptx::tmem_wait_ld();
          pair_columns(sv, dv, c0);
          if (kKeysHome) put_planes(sv, to, third);
          put_planes(dv, to + kDp, third + kDp);
        }
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      arrive_warp(&bars.p_full[kOneSlot ? 1 : i & 1]);
      row += kRows;
      if (--left == 0) {                                // the next head's queries
        row = first + kCols * w;
        left = per;
      }
      return true;
    };
    // three planes: the sums of step i, out of TMEM
    auto take = [&](int i) {
      if (!wait_warp(&bars.sum_full, i & 1)) return false;
      ptx::tc_fence_after();
      if constexpr (kPlanes == 3) add_columns(total, total_at);
      ptx::tc_fence_before();
      arrive_warp(&bars.sum_free);
      return true;
    };
    if (kPlanes == 1) {
      for (int i = 0; i < n && ok; ++i) ok = pairs(i);
    } else {
      for (int i = 0; i < n && ok; i += 2) {
        for (int j = i; j < i + 2 && j < n && ok; ++j) ok = pairs(j);
        for (int j = i; j < i + 2 && j < n && ok; ++j) ok = take(j);
      }
    }
    if (ok && n > 0) {
      ok = wait_warp(&bars.acc_full, 0);
      ptx::tc_fence_after();
    }
    if (!ok && lane == 0) report_timeout(status);
    const float nan = __uint_as_float(0x7FC00000u);
    auto put = [&](const Heads& t, uint32_t acc, float by, int cb0, int cb_step) {
      Out* p = static_cast<Out*>(t.p) + int64_t(b) * t.sb + int64_t(h) * t.sh + int64_t(r) * t.sl;
      const bool zero = n == 0 || (kKeysHome && r >= keys);
      for (int cb = cb0; cb < ksteps * 16; cb += cb_step) {
        uint32_t v[32];
        if constexpr (kPlanes == 3) {
          constexpr bool kTwo = kKeysHome;              // (of the thread's 64 or 32 sums)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(kTwo && cb == 32 ? total[kTwo ? 32 + e : e] : total[e]);
        } else if (n > 0) {
          ptx::tmem_ld32(tmem + lanes + acc + cb, v);
          ptx::tmem_wait_ld();
        }
        if (zero) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0u;
        }
        if (r < rows) store_columns(p, cb, a.dim, v, ok ? by : nan);
      }
    };
    if (kKeysHome) {
      if (w == 0) put(a.dv, kDv, 1.0f, 0, 32);
      else put(a.dk, kAcc, a.scale, 0, 32);
    } else {
      put(a.dq, kAcc, a.scale, 32 * w, 64);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (kPlanes == 1 && a.flags && threadIdx.x == 0)
    a.flags[(kKeysHome ? 0 : a.dq_flags) + (int64_t(b) * tiles + tile) * heads + h] = bars.bad;
  if (warp == 10) ptx::tmem_dealloc(tmem, kTmemCols);
}

// One launch for both: the first `key_blocks` blocks own keys, the others
// queries, which fill the SMs that the keys' blocks, uneven under a causal
// mask, leave early.
template <int kPlanes, bool kTma>
__global__ void __launch_bounds__(kThreads, 1)
    attention_tc_backward_kernel(AttentionArgs a, unsigned* status, const __grid_constant__ Maps key_maps,
                                 const __grid_constant__ Maps query_maps, unsigned key_blocks) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ BwdBars bars;
  if (blockIdx.x < key_blocks)
    backward_block<kPlanes, true, kTma>(a, status, key_maps.m, blockIdx.x, smem_raw, bars);
  else
    backward_block<kPlanes, false, kTma>(a, status, query_maps.m, blockIdx.x - key_blocks, smem_raw, bars);
}

size_t forward_smem(int planes, int dim) {
  const int stages = planes == 3 ? kFwdStages / 2 : kFwdStages;
  return 1024 + planes * (dim > 64 ? 2 : 1) * (2 * size_t(panel_bytes(128)) + stages * panel_bytes(kKeys));
}
size_t backward_smem(int planes, int dim) {
  return 1024 + planes * (dim > 64 ? 2 : 1) * size_t(2 * panel_bytes(128) + 2 * stages_of(planes) * panel_bytes(kStep));
}

template <typename K>
cudaError_t launch(PerDeviceOnce& once, K kernel, int64_t blocks, size_t smem, size_t most,
                   const AttentionArgs& a, const Maps& maps, cudaStream_t stream) {
  cudaError_t e = once.run([&](int) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  });
  if (e != cudaSuccess) return e;
  unsigned* status = nullptr;
  e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(a, status, maps);
  note_launch();
  return cudaGetLastError();
}

// Maps of a backward block's tensors; false where one is not one that TMA reads.
bool backward_maps(const AttentionArgs& a, bool keys_home, Maps& maps) {
  const int step = long_steps(a.bf16 ? 1 : 3) ? 2 * kStep : kStep;
  const int q_rows = keys_home ? step : 128, k_rows = keys_home ? 128 : step;
  const int q_at = keys_home ? 2 : 0, k_at = 2 - q_at;
  if (a.bf16)
    return make_map(&maps.m[q_at], a.q, a.batch, a.lq, a.hq, a.dim, q_rows) &&
           make_map(&maps.m[q_at + 1], a.dout, a.batch, a.lq, a.hq, a.dim, q_rows) &&
           make_map(&maps.m[k_at], a.k, a.batch, a.lk, a.hkv, a.dim, k_rows) &&
           make_map(&maps.m[k_at + 1], a.v, a.batch, a.lk, a.hkv, a.dim, k_rows);
  const int64_t n = 3 * int64_t(a.batch);
  return make_map(&maps.m[q_at], planes_of(a.planes[0], a.lq, a.hq, 64), n, a.lq, a.hq, 64, q_rows) &&
         make_map(&maps.m[q_at + 1], planes_of(a.planes[3], a.lq, a.hq, 64), n, a.lq, a.hq, 64, q_rows) &&
         make_map(&maps.m[k_at], planes_of(a.planes[1], a.lk, a.hkv, 64), n, a.lk, a.hkv, 64, k_rows) &&
         make_map(&maps.m[k_at + 1], planes_of(a.planes[2], a.lk, a.hkv, 64), n, a.lk, a.hkv, 64, k_rows);
}

template <int kPlanes, bool kTma>
cudaError_t launch_backward(const AttentionArgs& a, const Maps& key_maps, const Maps& query_maps, cudaStream_t stream) {
  static PerDeviceOnce once;
  const auto blocks = [](int64_t rows, int64_t heads, int64_t batch) {
    return (rows + kTcBackwardRows - 1) / kTcBackwardRows * heads * batch;
  };
  const int64_t key_blocks = a.dk.p ? blocks(a.lk, a.hkv, a.batch) : 0;
  const int64_t query_blocks = a.dq.p ? blocks(a.lq, a.hq, a.batch) : 0;
  if (key_blocks + query_blocks == 0) return cudaSuccess;
  const int most = static_cast<int>(backward_smem(kPlanes, kPlanes == 3 ? 64 : kMaxHeadDim));
  cudaError_t e = once.run([&](int) {
    return cudaFuncSetAttribute(attention_tc_backward_kernel<kPlanes, kTma>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  });
  if (e != cudaSuccess) return e;
  unsigned* status = nullptr;
  e = device_status_word(&status);
  if (e != cudaSuccess) return e;
  attention_tc_backward_kernel<kPlanes, kTma>
      <<<static_cast<unsigned>(key_blocks + query_blocks), kThreads, backward_smem(kPlanes, a.dim), stream>>>(
          a, status, key_maps, query_maps, static_cast<unsigned>(key_blocks));
  note_launch();
  return cudaGetLastError();
}

// The planes of q, k, v and, backward, dO (blockIdx.y): 8 columns per thread.
// Key rows past their length and values that a plane cannot hold become zero;
// for the latter the block's flag is set.  With dO a query's delta = do . o and
// lse2 are taken as well (a launch of their own took 6 of 129 us, f32 2 x 1024,
// 8 heads of 64, forward and backward).
__global__ void __launch_bounds__(256) attention_split_kernel(AttentionArgs a) {
  const int which = blockIdx.y;
  const Heads& t = which == 0 ? a.q : which == 1 ? a.k : which == 2 ? a.v : a.dout;
  const bool keyed = which == 1 || which == 2;
  const int length = keyed ? a.lk : a.lq, heads = keyed ? a.hkv : a.hq;
  const int64_t rows = int64_t(a.batch) * heads * length;
  const int width = a.dim > 64 ? 128 : 64, lanes = width / 8;     // threads per row
  const int64_t id = int64_t(blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  const int d = threadIdx.x % lanes * 8;
  bool bad = false;
  const int64_t rest = id / length;
  const int i = static_cast<int>(id - rest * length);
  const int b = static_cast<int>(rest / heads), h = static_cast<int>(rest - int64_t(b) * heads);
  float delta = 0.f;
  if (id < rows) {
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!keyed || i < keys_of(a, b)) {
      const float* p = static_cast<const float*>(t.p) + b * t.sb + h * t.sh + i * t.sl + d;
      if (d + 8 <= a.dim && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(p + e));
          f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (d + e < a.dim) f[e] = __ldg(p + e);
      }
    }
    if (which == 3) {
      float o[8];
      load8(static_cast<const float*>(a.o.p) + b * a.o.sb + h * a.o.sh + i * a.o.sl, d, a.dim, o);
      delta = dot8(f, o);
    }
    uint32_t w[3][4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (!(fabsf(f[e + j]) <= kMostSplit)) f[e + j] = 0.f, bad = true;
      uint32_t part[3];
      split_pair<3>(f[e], f[e + 1], part);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][e / 2] = part[q];
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4*>(static_cast<bf16*>(a.planes[which]) + ((q * rows + id) * width + d)) =
          make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
  }
  if (which == 3) {
    for (int o = lanes / 2; o > 0; o >>= 1) delta += __shfl_xor_sync(0xFFFFFFFFu, delta, o);
    if (id < rows && threadIdx.x % lanes == 0) {
      const int64_t at = rest * a.stat_stride;
      const float lse2 = __ldg(a.lse + id) * kLog2e;
      a.delta[at + i] = delta;
      a.lse2[at + i] = lse2 == -INFINITY ? INFINITY : lse2;
      if (i == length - 1)                                // the tile's rows past the last
        for (int j = length; j < a.stat_stride; ++j) {
          a.delta[at + j] = 0.f;
          a.lse2[at + j] = INFINITY;
        }
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.flags[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = bad;
}

}  // namespace

// A block's two halves hide one another's softmax, but where the blocks are so
// few that single halves all fit on the SMs at once, one half per block is
// done sooner (f32 4 x 1024, 4 heads of 64: 44 us against 64).
int attention_halves(const AttentionArgs& a) {
  return (int64_t(a.lq) + 127) / 128 * a.hq * a.batch <= 152 ? 1 : 2;
}

int64_t attention_split_blocks(const AttentionArgs& a) {
  const int64_t q = int64_t(a.batch) * a.hq * a.lq, k = int64_t(a.batch) * a.hkv * a.lk;
  const int64_t rows = a.dim > 64 ? 16 : 32;              // of a block
  return ((q > k ? q : k) + rows - 1) / rows;
}

cudaError_t launch_attention_split(const AttentionArgs& a, int tensors, cudaStream_t stream) {
  attention_split_kernel<<<dim3(static_cast<unsigned>(attention_split_blocks(a)), tensors), 256, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_attention_tc_forward(const AttentionArgs& a, cudaStream_t stream) {
  static PerDeviceOnce once, once_tma, once_split;
  const int64_t blocks = (int64_t(a.lq) + 128 * a.halves - 1) / (128 * a.halves) * a.hq * a.batch;
  Maps maps{};
  if (!a.bf16 && a.dim > 64) return launch_attention_wide_forward(a, stream);
  if (!a.bf16) {
    const size_t smem = forward_smem(3, a.dim);
    const int64_t n = 3 * int64_t(a.batch);
    if (!make_map(&maps.m[0], planes_of(a.planes[0], a.lq, a.hq, 64), n, a.lq, a.hq, 64, 128) ||
        !make_map(&maps.m[1], planes_of(a.planes[1], a.lk, a.hkv, 64), n, a.lk, a.hkv, 64, kKeys) ||
        !make_map(&maps.m[2], planes_of(a.planes[2], a.lk, a.hkv, 64), n, a.lk, a.hkv, 64, kKeys))
      return cudaErrorInvalidValue;
    return launch(once_split, attention_tc_forward_kernel<3, true>, blocks, smem, smem, a, maps, stream);
  }
  const size_t smem = forward_smem(1, a.dim), most = forward_smem(1, kMaxHeadDim);
  if (make_map(&maps.m[0], a.q, a.batch, a.lq, a.hq, a.dim, 128) &&
      make_map(&maps.m[1], a.k, a.batch, a.lk, a.hkv, a.dim, kKeys) &&
      make_map(&maps.m[2], a.v, a.batch, a.lk, a.hkv, a.dim, kKeys))
    return launch(once_tma, attention_tc_forward_kernel<1, true>, blocks, smem, most, a, maps, stream);
  return launch(once, attention_tc_forward_kernel<1, false>, blocks, smem, most, a, maps, stream);
}
cudaError_t launch_attention_tc_backward(const AttentionArgs& a, cudaStream_t stream) {
  if (!a.bf16 && a.dim > 64) return launch_attention_wide_backward(a, stream);
  Maps key_maps{}, query_maps{};
  const bool tma = backward_maps(a, true, key_maps) && backward_maps(a, false, query_maps);
  if (!a.bf16)
    return tma ? launch_backward<3, true>(a, key_maps, query_maps, stream) : cudaErrorInvalidValue;
  return tma ? launch_backward<1, true>(a, key_maps, query_maps, stream)
             : launch_backward<1, false>(a, key_maps, query_maps, stream);
}

}  // namespace det
