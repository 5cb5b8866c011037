// Differential attention, backward (the formulas stand in diff_shared.cuh).
// No atomics: two runs on the same inputs give the same bits.
//  1. diff_rows_kernel: Delta_m and -LSE_m log2(e) of every query row, and the
//     sum of Delta_2 over 64 rows, the summands of dlambda.
//  2. diff_dlambda_kernel: dlambda_h from those sums, in a fixed order.
//  3. diff_dkdv_kernel, key-tile-major: 128 keys against steps of 64 queries.
//  4. diff_dq_kernel, query-tile-major: 128 queries against steps of 64 keys.
//
// Both matrix kernels run on the tensor cores with a step of 64 columns, so that
// two steps fit into TMEM next to the accumulators and one warpgroup works on
// each: while warpgroup 0 takes the exponentials of step g, the tensor cores run
// the products of step g + 1 for warpgroup 1, and the other way round.  The maps
// share dA = dO V^T, and both maps' probabilities enter dV in one product, so
// the products cost what plain attention's backward costs; the exponentials are
// twice as many.
#include "diff_shared.cuh"

namespace uaa {
namespace {

constexpr int kStep = 64;  // queries (dK/dV) or keys (dQ) of a step
constexpr int kThreads = 320;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kStepChunk = kStep * 128;  // 64 rows x 128 bytes: 64 columns of a step's operand

__host__ __device__ __forceinline__ int steps_of(int S) { return 2 * tiles_of(S); }
// Row vectors, (B, H, steps, 4, 64): -LSE_1 log2(e), -LSE_2 log2(e), Delta_1, Delta_2 of a step's queries
__host__ __device__ __forceinline__ size_t rows_at(size_t bh, int Sq, int i) {
  return (bh * steps_of(Sq) + i / kStep) * (4 * kStep) + i % kStep;
}

// 16 / 8 packed columns of this thread's TMEM lane, then a wait for the store.
__device__ __forceinline__ void tmem_st16_bits(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8_bits(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v, float c) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0] * c, v[1] * c), pack_bf16(v[2] * c, v[3] * c),
                                            pack_bf16(v[4] * c, v[5] * c), pack_bf16(v[6] * c, v[7] * c));
}

// ---------------------------------------------------------------------------
// 1. Row vectors.  A block takes 64 rows of kRowHeads heads: D/8 lanes of 16 bytes a row, the heads in turn, so
// that neighbouring reads follow each other and a head's results are written as runs.
constexpr int kRowThreads = 256;
constexpr int kRowHeads = 4;

template <int D>
__global__ void __launch_bounds__(kRowThreads) diff_rows_kernel(
    const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ out2,
    const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse, const void* __restrict__ lam, int lam_bf16,
    float* __restrict__ rows, float* __restrict__ part, int B, int Sq, int H) {
  constexpr int G = D / 8;
  constexpr int kGroups = kRowThreads / G;
  __shared__ float sums[kGroups];
  const int group = threadIdx.x / G, sub = threadIdx.x % G;
  const int steps = steps_of(Sq), hgroups = (H + kRowHeads - 1) / kRowHeads;
  const long long unit = blockIdx.x;
  const int h0 = (int)(unit % hgroups) * kRowHeads;
  const int t = (int)(unit / hgroups % steps), b = (int)(unit / hgroups / steps);
  for (int h = h0; h < min(H, h0 + kRowHeads); ++h) {
    const size_t bh = (size_t)b * H + h;
    const float lm = load_lambda(lam, lam_bf16, h);
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < kStep / kGroups; ++r) {
      const int i = t * kStep + r * kGroups + group;
      float d1 = 0.f, d2 = 0.f;
      if (i < Sq) {
        const size_t at = (((size_t)b * Sq + i) * H + h) * D + 8 * sub;
        const uint4 o = __ldg(reinterpret_cast<const uint4*>(out + at));
        const uint4 p = __ldg(reinterpret_cast<const uint4*>(out2 + at));
        const uint4 g = __ldg(reinterpret_cast<const uint4*>(dout + at));
        const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&o);
        const __nv_bfloat162* p2 = reinterpret_cast<const __nv_bfloat162*>(&p);
        const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 of = __bfloat1622float2(o2[e]), pf = __bfloat1622float2(p2[e]), gf = __bfloat1622float2(g2[e]);
          d1 = fmaf(of.x, gf.x, fmaf(of.y, gf.y, d1));
          d2 = fmaf(pf.x, gf.x, fmaf(pf.y, gf.y, d2));
        }
      }
#pragma unroll
      for (int o = G / 2; o > 0; o /= 2) {
        d1 += __shfl_xor_sync(0xffffffffu, d1, o);
        d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      }
      sum += d2;
      if (sub < 4) {
        float x = sub == 2 ? fmaf(lm, d2, d1) : d2;
        if (sub < 2) {
          const float l = i < Sq ? lse[(bh * 2 + sub) * Sq + i] : -INFINITY;
          x = l == -INFINITY ? -INFINITY : -l * kLog2e;  // rows past Sq, or without a key: P = 0
        }
        rows[rows_at(bh, Sq, i) + sub * kStep] = x;
      }
    }
    if (sub == 0) sums[group] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.f;
      for (int x = 0; x < kGroups; ++x) s += sums[x];
      part[(size_t)h * B * steps + (size_t)b * steps + t] = s;
    }
    __syncthreads();
  }
}

// 2. dlambda_h = -sum of Delta_2 over the head's rows, one block per head.
__global__ void __launch_bounds__(256) diff_dlambda_kernel(const float* __restrict__ part, void* __restrict__ dlam,
                                                           int lam_bf16, int n) {
  __shared__ float sums[8];
  const int h = blockIdx.x;
  float s = 0.f;
  for (int i = threadIdx.x; i < n; i += 256) s += part[(size_t)h * n + i];
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int x = 0; x < 8; ++x) s += sums[x];
    if (lam_bf16)
      static_cast<__nv_bfloat16*>(dlam)[h] = __float2bfloat16_rn(-s);
    else
      static_cast<float*>(dlam)[h] = -s;
  }
}

struct Item {
  int t, h, b;
};
__device__ __forceinline__ Item decode_item(int item, int tiles, int H, bool head_inner) {
  Item it;
  if (head_inner) {
    it.h = item % H;
    it.t = item / H % tiles;
    it.b = item / H / tiles;
  } else {
    it.t = item % tiles;
    it.h = item / tiles % H;
    it.b = item / tiles / H;
  }
  return it;
}

// ---------------------------------------------------------------------------
// 3. dK, dV.  A persistent CTA takes 128 keys of one (batch, head) and loops over steps of 64 queries:
//     S_m^T = K_m Q_m^T, P^T = A_1^T - lambda A_2^T, dA^T = V dO^T       (M = keys, N = 64)
//     dV += P^T dO, dK_m += dS_m^T Q_m
// TMEM, per step parity 128 columns: X holds S_1^T, then P^T (32 packed columns) and dS_2^T (columns 32..63);
// Y holds S_2^T, then dA^T (formed once both S have been read), then dS_1^T.  dV is at 256, dK_m at 384 + 64 m
// (64 columns each; with D = 64 the product runs over all 64 columns of Q and map m's 32 are kept).
// One elected lane issues, per step g: dA_g dV_g after p_ready(g), dK_g S_{g+2} after ds_ready(g).
// MMAs of one thread run in order, but two that read A from TMEM for different products are only relied on
// with equal shapes: dV_g (N = D) has completed before dK_g (N = 64) is issued.
template <int D>
struct DkdvLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStepBytes = kStep * D * 2;
  static constexpr int kRing = D == 128 ? 4 : 6;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQ = kV + kTileBytes;           // Q steps, then dO steps, then row vectors
  static constexpr int kDO = kQ + kRing * kStepBytes;
  static constexpr int kRows = kDO + kRing * kStepBytes;
  static constexpr int kCtl = kRows + kRing * 4 * kStep * 4;
  static constexpr int kSmem = kCtl + 256;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

struct DkdvCtl {
  uint64_t bar_kv_full, bar_kv_empty;
  uint64_t bar_full[6], bar_empty[6];
  uint64_t bar_s_full[2], bar_dp_full[2], bar_p_ready[2], bar_ds_ready[2];
  uint64_t bar_dv_done, bar_acc_done, bar_acc_free, bar_final;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DkdvCtl) <= 256, "control block");

// Is any key of tile t attended?  (warp-collective)
__device__ __forceinline__ bool tile_any(const uint8_t* __restrict__ mask, int b, int t, int Sk) {
  const int lane = threadIdx.x & 31;
  bool hit = false;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int j = t * kTile + 32 * x + lane;
    hit |= j < Sk && mask[(size_t)b * Sk + j] != 0;
  }
  return __any_sync(0xffffffffu, hit);
}

template <int D, bool kMask>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const void* __restrict__ lam, int lam_bf16, const float* __restrict__ rows,
                     const uint8_t* __restrict__ key_mask, __nv_bfloat16* __restrict__ dk,
                     __nv_bfloat16* __restrict__ dv, int B, int H, int Sq, int Sk, int num_items, int head_inner,
                     float scale, float scale_log2, DevCtx ctx) {
  using L = DkdvLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, kStep, false, false);  // S^T, dA^T
  constexpr uint32_t kIdescV = idesc_bf16_f32(128, D, false, true);       // dV (A in TMEM)
  constexpr uint32_t kIdescK = idesc_bf16_f32(128, 64, false, true);      // dK_m (A in TMEM)
  constexpr uint32_t kX = 0, kY = 64, kStage = 128, kColDV = 256, kColDK = 384;

  extern __shared__ __align__(1024) uint8_t smem[];
  DkdvCtl* ctl = reinterpret_cast<DkdvCtl*>(smem + L::kCtl);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nkt = tiles_of(Sk);
  const int n = (Sq + kStep - 1) / kStep;  // steps of an item

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_kv_full, 1);
    mbar_init(&ctl->bar_kv_empty, 1);
    for (int s = 0; s < R; ++s) {
      mbar_init(&ctl->bar_full[s], 1);
      mbar_init(&ctl->bar_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->bar_s_full[s], 1);
      mbar_init(&ctl->bar_dp_full[s], 1);
      mbar_init(&ctl->bar_p_ready[s], 128);
      mbar_init(&ctl->bar_ds_ready[s], 128);
    }
    mbar_init(&ctl->bar_dv_done, 1);
    mbar_init(&ctl->bar_acc_done, 1);
    mbar_init(&ctl->bar_acc_free, 256);
    mbar_init(&ctl->bar_final, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDO);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t k_extent = (size_t)B * Sk * H * D;

  uint32_t armed[6] = {}, kv_armed = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t G = 0, it = 0;  // steps and items so far
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nkt, H, head_inner);
      if (kMask && !tile_any(key_mask, w.b, w.t, Sk)) continue;
      if (lane == 0) {
        if (it > 0) ok = wait_or_abort(&ctl->bar_kv_empty, (it - 1) & 1, ctx, ctl);
        if (ok) {
          mbar_arrive_expect_tx(&ctl->bar_kv_full, 2 * L::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kK + c * kChunkBytes, &tmK, &ctl->bar_kv_full, c * 64, w.h, w.t * kTile, w.b);
            tma_load_4d(smem + L::kV + c * kChunkBytes, &tmV, &ctl->bar_kv_full, c * 64, w.h, w.t * kTile, w.b);
          }
          kv_armed = it + 1;
        }
        const float* rsrc = rows + rows_at((size_t)w.b * H + w.h, Sq, 0);
        for (int g = 0; ok && g < n; ++g, ++G) {
          const int slot = G % R;
          const uint32_t use = G / R;
          if (use > 0) ok = wait_or_abort(&ctl->bar_empty[slot], (use - 1) & 1, ctx, ctl);
          if (!ok) break;
          if ((int)G == ctx.drop_load) continue;
          mbar_arrive_expect_tx(&ctl->bar_full[slot], 2 * L::kStepBytes + 4 * kStep * 4);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kQ + slot * L::kStepBytes + c * kStepChunk, &tmQ, &ctl->bar_full[slot], c * 64, w.h,
                        g * kStep, w.b);
            tma_load_4d(smem + L::kDO + slot * L::kStepBytes + c * kStepChunk, &tmDO, &ctl->bar_full[slot], c * 64,
                        w.h, g * kStep, w.b);
          }
          bulk_load(smem + L::kRows + slot * 4 * kStep * 4, rsrc + (size_t)g * 4 * kStep, 4 * kStep * 4,
                    &ctl->bar_full[slot]);
          armed[slot] = use + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++it;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t el_lane;
    const bool el = elect_one_sync(&el_lane);
    bool ok = true;
    uint32_t G0 = 0, it = 0;
    auto wait_el = [&](uint64_t* bar, uint32_t parity) {
      bool w = true;
      if (el) w = wait_or_abort(bar, parity, ctx, ctl);
      return __shfl_sync(0xffffffffu, w ? 1 : 0, el_lane) != 0;
    };
    auto sq = [&](uint32_t G) { return sbase + L::kQ + (G % R) * L::kStepBytes; };
    auto sdo = [&](uint32_t G) { return sbase + L::kDO + (G % R) * L::kStepBytes; };
    // 16-column step kk of a 64-row operand of D columns
    auto step_off = [](int kk) { return (uint32_t)((kk >> 2) * kStepChunk + (kk & 3) * 32); };
    auto tile_off = [](int kk) { return (uint32_t)((kk >> 2) * kChunkBytes + (kk & 3) * 32); };
    auto issue_s = [&](uint32_t G) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kK, 16, 1024), b0 = sdesc_sw128(sq(G), 16, 1024);
      const uint32_t d = tmem + (G & 1) * kStage;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int m = kk >= D / 32;
        const uint64_t a = desc_add(a0, tile_off(kk)), b = desc_add(b0, step_off(kk));
        if (el) mma_ss_checked(mg, d + (m ? kY : kX), a, b, kIdescS, kk % (D / 32) > 0, kStep);
      }
      if (el) mma_commit(&ctl->bar_s_full[G & 1]);
    };
    auto issue_dp = [&](uint32_t G) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kV, 16, 1024), b0 = sdesc_sw128(sdo(G), 16, 1024);
      const uint32_t d = tmem + (G & 1) * kStage + kY;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t a = desc_add(a0, tile_off(kk)), b = desc_add(b0, step_off(kk));
        if (el) mma_ss_checked(mg, d, a, b, kIdescS, kk > 0, kStep);
      }
      if (el) mma_commit(&ctl->bar_dp_full[G & 1]);
    };
    auto issue_dv = [&](uint32_t G, bool first) {
      const uint64_t b0 = sdesc_sw128(sdo(G), kStepChunk, 1024);
      const uint32_t a = tmem + (G & 1) * kStage + kX;
#pragma unroll
      for (int kk = 0; kk < kStep / 16; ++kk) {
        const uint64_t b = desc_add(b0, kk * 2048);
        if (el) mma_ts_checked(mg, tmem + kColDV, a + kk * 8, b, kIdescV, (!first || kk > 0) ? 1u : 0u, D);
      }
      if (el) mma_commit(&ctl->bar_dv_done);
    };
    auto issue_dk = [&](uint32_t G, bool first) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint64_t b0 = sdesc_sw128(sq(G) + (D == 128 ? m * kStepChunk : 0), kStepChunk, 1024);
        const uint32_t a = tmem + (G & 1) * kStage + (m ? kX + 32 : kY);
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk) {
          const uint64_t b = desc_add(b0, kk * 2048);
          if (el)
            mma_ts_checked(mg, tmem + kColDK + 64 * m, a + kk * 8, b, kIdescK, (!first || kk > 0) ? 1u : 0u, 64);
        }
      }
      if (el) mma_commit(&ctl->bar_empty[G % R]);
    };
    auto full = [&](uint32_t G) { return wait_el(&ctl->bar_full[G % R], (G / R) & 1); };
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nkt, H, head_inner);
      if (kMask && !tile_any(key_mask, w.b, w.t, Sk)) continue;
      ok = wait_el(&ctl->bar_kv_full, it & 1);
      for (int g = 0; ok && g < 2 && g < n; ++g) {
        if (!(ok = full(G0 + g))) break;
        tc_fence_after();
        issue_s(G0 + g);
        if (el) mma_issued = true;
      }
      for (int g = 0; ok && g < n; ++g) {
        const uint32_t G = G0 + g, st = G & 1, ph = (G >> 1) & 1;
        if (!(ok = wait_el(&ctl->bar_p_ready[st], ph))) break;
        // the previous item's epilogue must have read dV and dK
        if (g == 0 && it > 0 && !(ok = wait_el(&ctl->bar_acc_free, (it - 1) & 1))) break;
        tc_fence_after();
        issue_dp(G);
        issue_dv(G, g == 0);
        if (!(ok = wait_el(&ctl->bar_ds_ready[st], ph))) break;
        if (!(ok = wait_el(&ctl->bar_dv_done, G & 1))) break;
        tc_fence_after();
        issue_dk(G, g == 0);
        if (g + 2 < n) {
          if (!(ok = full(G + 2))) break;
          tc_fence_after();
          issue_s(G + 2);
        }
      }
      if (el) {
        if (ok) {
          mma_commit(&ctl->bar_acc_done);
          mma_commit(&ctl->bar_kv_empty);
        } else {
          *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        }
      }
      __syncwarp();
      G0 += n;
      ++it;
    }
  } else {
    // ------------------------------------------------------------ compute: warpgroup wg takes steps of its parity
    const int wg = warp >> 2;
    const int jrow = (warp & 3) * 32 + lane;  // key row = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tX = tl + wg * kStage + kX, tY = tl + wg * kStage + kY;
    bool ok = true;
    uint32_t G0 = 0, it = 0;
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nkt, H, head_inner);
      const int j = w.t * kTile + jrow;
      const bool exists = j < Sk;
      // this thread writes half of the row's columns: half wg
      const size_t off = (((size_t)w.b * Sk + (exists ? j : 0)) * H + w.h) * D + wg * (D / 2);
      const bool store = exists && guard_store(ctx, off, D / 2, k_extent);
      if (kMask && !tile_any(key_mask, w.b, w.t, Sk)) {
        // no attended key in this tile: dK = dV = 0
        if (store) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            *reinterpret_cast<uint4*>(dk + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(dv + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      const bool attended = exists && (!kMask || key_mask[(size_t)w.b * Sk + j] != 0);
      const float neg_lam = -load_lambda(lam, lam_bf16, w.h);
      const float2 nl = make_float2(neg_lam, neg_lam), c2 = make_float2(scale_log2, scale_log2);
      for (int g = 0; g < n; ++g) {
        const uint32_t G = G0 + g, ph = (G >> 1) & 1;
        if ((G & 1) != (uint32_t)wg) continue;
        const float* rv = reinterpret_cast<const float*>(smem + L::kRows + (G % R) * 4 * kStep * 4);
        bool okw = wait_or_abort(&ctl->bar_full[G % R], (G / R) & 1, ctx, ctl);
        if (okw) okw = wait_or_abort(&ctl->bar_s_full[wg], ph, ctx, ctl);
        if (!(ok = __all_sync(0xffffffffu, okw))) break;
        tc_fence_after();
        float p1[kStep], p2[kStep];  // A_1 and -lambda A_2
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s[64];
          tmem_ld32x2(tX + 32 * c, tY + 32 * c, s);
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int q = 32 * c + 2 * i;
            const float2 x1 = fma2(make_float2(s[2 * i], s[2 * i + 1]), c2, *reinterpret_cast<const float2*>(rv + q));
            const float2 x2 = fma2(make_float2(s[32 + 2 * i], s[33 + 2 * i]), c2,
                                   *reinterpret_cast<const float2*>(rv + kStep + q));
            const float2 a = make_float2(ex2(x1.x), ex2(x1.y));
            const float2 b = mul2(make_float2(ex2(x2.x), ex2(x2.y)), nl);
            p1[q] = a.x, p1[q + 1] = a.y, p2[q] = b.x, p2[q + 1] = b.y;
            pk[i] = pack_bf16(a.x + b.x, a.y + b.y);
          }
          tmem_st16_bits(tX + 16 * c, pk);  // P^T, over columns of S_1^T that were read
        }
        tc_fence_before();
        mbar_arrive(&ctl->bar_p_ready[wg]);
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dp_full[wg], ph, ctx, ctl)))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float dp[16];
          tmem_ld16(tY + 16 * c, dp);
          uint32_t k1[8], k2[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int q = 16 * c + 2 * i;
            const float2 d = make_float2(dp[2 * i], dp[2 * i + 1]);
            const float2 a = mul2(make_float2(p1[q], p1[q + 1]),
                                  sub2(d, *reinterpret_cast<const float2*>(rv + 2 * kStep + q)));
            const float2 b = mul2(make_float2(p2[q], p2[q + 1]),
                                  sub2(d, *reinterpret_cast<const float2*>(rv + 3 * kStep + q)));
            k1[i] = pack_bf16(a.x, a.y);
            k2[i] = pack_bf16(b.x, b.y);
          }
          tmem_st8_bits(tY + 8 * c, k1);        // dS_1^T, over columns of dA^T that were read
          tmem_st8_bits(tX + 32 + 8 * c, k2);   // dS_2^T, beside P^T
        }
        tc_fence_before();
        mbar_arrive(&ctl->bar_ds_ready[wg]);
      }
      if (!ok) break;
      G0 += n;
      // epilogue: dV, and dK = scale * (dS^T Q).  A key outside the mask gets zeros, whatever its rows hold.
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_acc_done, it & 1, ctx, ctl)))) break;
      tc_fence_after();
      const uint32_t cV = tl + kColDV + wg * (D / 2), cK = tl + kColDK + 64 * wg + (D == 64 ? 32 * wg : 0);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        float gv[64];
        tmem_ld32x2(cV + 32 * c, cK + 32 * c, gv);
        if (!attended) {
#pragma unroll
          for (int i = 0; i < 64; ++i) gv[i] = 0.f;
        }
        if (store) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            store8(dv + off + 32 * c + 8 * i, gv + 8 * i, 1.f);
            store8(dk + off + 32 * c + 8 * i, gv + 32 + 8 * i, scale);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&ctl->bar_acc_free);
      ++it;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp && mma_issued) {
    mma_commit(&ctl->bar_final);
    settle(&ctl->bar_final, 0, ctx);
  }
  if (warp == kProducerWarp && lane == 0) {
    if (kv_armed) settle(&ctl->bar_kv_full, (kv_armed - 1) & 1, ctx);
    for (int s = 0; s < R; ++s)
      if (armed[s]) settle(&ctl->bar_full[s], (armed[s] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// 4. dQ.  A persistent CTA takes 128 queries of one (batch, head), Q and dO in shared memory, and loops over steps
// of 64 keys: S_m = Q_m K_m^T, dA = dO V^T (M = queries, N = 64), then dQ_m += dS_m K_m.
// TMEM, per step parity 192 columns: S_1 (then dS_1), S_2 (then dS_2), dA; dQ_m at 384 + 64 m (with D = 64 the
// product runs over all 64 columns of K and map m's 32 are kept).  One elected lane issues dQ_g and the three
// products of step g + 2 after ds_ready(g).
template <int D>
struct DqLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStepBytes = kStep * D * 2;
  static constexpr int kRing = D == 128 ? 5 : 8;
  static constexpr int kQ = 0;
  static constexpr int kDO = kQ + kTileBytes;
  static constexpr int kK = kDO + kTileBytes;
  static constexpr int kV = kK + kRing * kStepBytes;
  static constexpr int kCtl = kV + kRing * kStepBytes;
  static constexpr int kCnt = kCtl + 384;  // attended steps per mask row
  static constexpr int kSmem = kCnt + kMaxCntRows * 4;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

struct DqCtl {
  uint64_t bar_q_full, bar_q_empty;
  uint64_t bar_full[8], bar_empty[8];
  uint64_t bar_s_full[2], bar_ds_ready[2];
  uint64_t bar_dq_done, bar_dq_free, bar_final;
  uint32_t tmem_base;
  int abort;
  uint32_t mask_words[8][2];  // per ring slot: the attended keys of its step
};
static_assert(sizeof(DqCtl) <= 384, "control block");

template <int D, bool kMask>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const void* __restrict__ lam, int lam_bf16, const float* __restrict__ rows,
                   const uint8_t* __restrict__ key_mask, __nv_bfloat16* __restrict__ dq, int B, int H, int Sq, int Sk,
                   int num_items, float scale, float scale_log2, DevCtx ctx) {
  using L = DqLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, kStep, false, false);  // S, dA
  constexpr uint32_t kIdescQ = idesc_bf16_f32(128, 64, false, true);      // dQ_m (A in TMEM)
  constexpr uint32_t kStage = 192, kColDP = 128, kColDQ = 384;

  extern __shared__ __align__(1024) uint8_t smem[];
  DqCtl* ctl = reinterpret_cast<DqCtl*>(smem + L::kCtl);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nqt = tiles_of(Sq);
  const int nks = (Sk + kStep - 1) / kStep;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_q_full, 1);
    mbar_init(&ctl->bar_q_empty, 1);
    for (int s = 0; s < R; ++s) {
      mbar_init(&ctl->bar_full[s], 1);
      mbar_init(&ctl->bar_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->bar_s_full[s], 1);
      mbar_init(&ctl->bar_ds_ready[s], 128);
    }
    mbar_init(&ctl->bar_dq_done, 1);
    mbar_init(&ctl->bar_dq_free, 256);
    mbar_init(&ctl->bar_final, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDO);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  // Attended steps per mask row: every role takes its step count from this table, which no one writes after the
  // start; only the producer reads the mask itself and leaves each step's bits with its ring slot.
  int* step_cnt = reinterpret_cast<int*>(smem + L::kCnt);
  const bool skip = kMask && B <= kMaxCntRows;
  if (skip) {
    for (int r = threadIdx.x; r < B; r += kThreads) step_cnt[r] = 0;
    __syncthreads();
    const int pairs = B * nks;
    for (int p0 = warp * 4; p0 < pairs; p0 += (kThreads / 32) * 4) {
      bool any[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pr = p0 + u;
        bool hit = false;
        if (pr < pairs) {
          const int r = pr / nks, k0 = (pr - r * nks) * kStep;
          const uint8_t* row = key_mask + (size_t)r * Sk + k0;
          hit = (k0 + lane < Sk && row[lane] != 0) || (k0 + 32 + lane < Sk && row[32 + lane] != 0);
        }
        any[u] = hit;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (__any_sync(0xffffffffu, any[u]) && lane == 0 && p0 + u < pairs) atomicAdd(&step_cnt[(p0 + u) / nks], 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t q_extent = (size_t)B * Sq * H * D;
  auto item_steps = [&](int b) { return skip ? step_cnt[b] : nks; };

  uint32_t armed[8] = {}, q_armed = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t G = 0, it = 0;
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H, false);
      if (item_steps(w.b) == 0) continue;  // no attended key: the compute warps write dQ = 0
      if (lane == 0) {
        if (it > 0) ok = wait_or_abort(&ctl->bar_q_empty, (it - 1) & 1, ctx, ctl);
        if (ok) {
          mbar_arrive_expect_tx(&ctl->bar_q_full, 2 * L::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kQ + c * kChunkBytes, &tmQ, &ctl->bar_q_full, c * 64, w.h, w.t * kTile, w.b);
            tma_load_4d(smem + L::kDO + c * kChunkBytes, &tmDO, &ctl->bar_q_full, c * 64, w.h, w.t * kTile, w.b);
          }
          q_armed = it + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++it;
      for (int j = 0; ok && j < nks; ++j) {
        uint32_t words[2] = {0u, 0u};
        if (kMask) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int c = j * kStep + 32 * t + lane;
            words[t] = __ballot_sync(0xffffffffu, c < Sk && key_mask[(size_t)w.b * Sk + c] != 0);
          }
          if (skip && (words[0] | words[1]) == 0) continue;
        }
        const int slot = G % R;
        const uint32_t use = G / R;
        if (lane == 0) {
          if (use > 0) ok = wait_or_abort(&ctl->bar_empty[slot], (use - 1) & 1, ctx, ctl);
          if (ok) {
            ctl->mask_words[slot][0] = words[0];
            ctl->mask_words[slot][1] = words[1];
            if ((int)G != ctx.drop_load) {
              mbar_arrive_expect_tx(&ctl->bar_full[slot], 2 * L::kStepBytes);
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                tma_load_4d(smem + L::kK + slot * L::kStepBytes + c * kStepChunk, &tmK, &ctl->bar_full[slot], c * 64,
                            w.h, j * kStep, w.b);
                tma_load_4d(smem + L::kV + slot * L::kStepBytes + c * kStepChunk, &tmV, &ctl->bar_full[slot], c * 64,
                            w.h, j * kStep, w.b);
              }
              armed[slot] = use + 1;
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++G;
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t el_lane;
    const bool el = elect_one_sync(&el_lane);
    bool ok = true;
    uint32_t G0 = 0, it = 0;
    auto wait_el = [&](uint64_t* bar, uint32_t parity) {
      bool w = true;
      if (el) w = wait_or_abort(bar, parity, ctx, ctl);
      return __shfl_sync(0xffffffffu, w ? 1 : 0, el_lane) != 0;
    };
    auto sk = [&](uint32_t G) { return sbase + L::kK + (G % R) * L::kStepBytes; };
    auto sv = [&](uint32_t G) { return sbase + L::kV + (G % R) * L::kStepBytes; };
    auto step_off = [](int kk) { return (uint32_t)((kk >> 2) * kStepChunk + (kk & 3) * 32); };
    auto tile_off = [](int kk) { return (uint32_t)((kk >> 2) * kChunkBytes + (kk & 3) * 32); };
    // S_1, S_2 and dA of step G
    auto issue_kk = [&](uint32_t G) {
      const uint32_t d = tmem + (G & 1) * kStage;
      const uint64_t a0 = sdesc_sw128(sbase + L::kQ, 16, 1024), b0 = sdesc_sw128(sk(G), 16, 1024);
      const uint64_t a1 = sdesc_sw128(sbase + L::kDO, 16, 1024), b1 = sdesc_sw128(sv(G), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int m = kk >= D / 32;
        const uint64_t a = desc_add(a0, tile_off(kk)), b = desc_add(b0, step_off(kk));
        if (el) mma_ss_checked(mg, d + (m ? 64 : 0), a, b, kIdescS, kk % (D / 32) > 0, kStep);
      }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t a = desc_add(a1, tile_off(kk)), b = desc_add(b1, step_off(kk));
        if (el) mma_ss_checked(mg, d + kColDP, a, b, kIdescS, kk > 0, kStep);
      }
      if (el) mma_commit(&ctl->bar_s_full[G & 1]);
    };
    auto issue_dq = [&](uint32_t G, bool first) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint64_t b0 = sdesc_sw128(sk(G) + (D == 128 ? m * kStepChunk : 0), kStepChunk, 1024);
        const uint32_t a = tmem + (G & 1) * kStage + 64 * m;
#pragma unroll
        for (int kk = 0; kk < kStep / 16; ++kk) {
          const uint64_t b = desc_add(b0, kk * 2048);
          if (el)
            mma_ts_checked(mg, tmem + kColDQ + 64 * m, a + kk * 8, b, kIdescQ, (!first || kk > 0) ? 1u : 0u, 64);
        }
      }
      if (el) mma_commit(&ctl->bar_empty[G % R]);
    };
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H, false);
      const int n = item_steps(w.b);
      if (n == 0) continue;
      ok = wait_el(&ctl->bar_q_full, it & 1);
      for (int g = 0; ok && g < 2 && g < n; ++g) {
        if (!(ok = wait_el(&ctl->bar_full[(G0 + g) % R], ((G0 + g) / R) & 1))) break;
        tc_fence_after();
        issue_kk(G0 + g);
        if (el) mma_issued = true;
      }
      if (ok && el && n <= 2) mma_commit(&ctl->bar_q_empty);
      for (int g = 0; ok && g < n; ++g) {
        const uint32_t G = G0 + g;
        if (!(ok = wait_el(&ctl->bar_ds_ready[G & 1], (G >> 1) & 1))) break;
        // the previous item's epilogue must have read dQ
        if (g == 0 && it > 0 && !(ok = wait_el(&ctl->bar_dq_free, (it - 1) & 1))) break;
        tc_fence_after();
        issue_dq(G, g == 0);
        if (g + 2 < n) {
          if (!(ok = wait_el(&ctl->bar_full[(G + 2) % R], ((G + 2) / R) & 1))) break;
          tc_fence_after();
          issue_kk(G + 2);
          if (el && g + 3 == n) mma_commit(&ctl->bar_q_empty);  // the item's last products with Q and dO
        }
      }
      if (el) {
        if (ok)
          mma_commit(&ctl->bar_dq_done);
        else
          *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
      }
      __syncwarp();
      G0 += n;
      ++it;
    }
  } else {
    // ------------------------------------------------------------ compute: warpgroup wg takes steps of its parity
    const int wg = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // query row = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + wg * kStage;
    bool ok = true;
    uint32_t G0 = 0, it = 0;
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H, false);
      const int n = item_steps(w.b);
      const int i = w.t * kTile + row;
      // this thread writes half of the row's columns: map wg's
      const size_t off = (((size_t)w.b * Sq + (i < Sq ? i : 0)) * H + w.h) * D + wg * (D / 2);
      const bool store = i < Sq && guard_store(ctx, off, D / 2, q_extent);
      if (n == 0) {
        if (store) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) *reinterpret_cast<uint4*>(dq + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const float* rv = rows + rows_at((size_t)w.b * H + w.h, Sq, i);  // rows past Sq: -inf and 0
      const float n1 = rv[0], n2 = rv[kStep], d1 = rv[2 * kStep], d2 = rv[3 * kStep];
      const float neg_lam = -load_lambda(lam, lam_bf16, w.h);
      const float2 c2 = make_float2(scale_log2, scale_log2), nl = make_float2(neg_lam, neg_lam);
      for (int g = 0; g < n; ++g) {
        const uint32_t G = G0 + g;
        if ((G & 1) != (uint32_t)wg) continue;
        const int slot = G % R;
        bool okw = wait_or_abort(&ctl->bar_full[slot], (G / R) & 1, ctx, ctl);
        if (okw) okw = wait_or_abort(&ctl->bar_s_full[wg], (G >> 1) & 1, ctx, ctl);
        if (!(ok = __all_sync(0xffffffffu, okw))) break;
        tc_fence_after();
        uint32_t words[2] = {0xffffffffu, 0xffffffffu};
        if (kMask) {
          words[0] = ctl->mask_words[slot][0];
          words[1] = ctl->mask_words[slot][1];
        } else if (g == n - 1 && Sk % kStep) {  // keys past the end
          const int left = Sk % kStep;
          words[0] = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
          words[1] = left > 32 ? (1u << (left - 32)) - 1u : 0u;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s[64], dp[32];
          tmem_ld32x2(tS + 32 * c, tS + 64 + 32 * c, s);
          tmem_ld32(tS + kColDP + 32 * c, dp);
          uint32_t k1[16], k2[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float2 x1 = fma2(make_float2(s[2 * x], s[2 * x + 1]), c2, make_float2(n1, n1));
            const float2 x2 = fma2(make_float2(s[32 + 2 * x], s[33 + 2 * x]), c2, make_float2(n2, n2));
            const float2 d = make_float2(dp[2 * x], dp[2 * x + 1]);
            float2 a = mul2(make_float2(ex2(x1.x), ex2(x1.y)), sub2(d, make_float2(d1, d1)));
            float2 b = mul2(mul2(make_float2(ex2(x2.x), ex2(x2.y)), nl), sub2(d, make_float2(d2, d2)));
            s[2 * x] = a.x, s[2 * x + 1] = a.y, s[32 + 2 * x] = b.x, s[33 + 2 * x] = b.y;
          }
          if (words[c] != 0xffffffffu) {
            // keys outside the mask, or past the end: dS = 0 whatever their rows hold
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((words[c] >> x) & 1u)) s[x] = s[32 + x] = 0.f;
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            k1[x] = pack_bf16(s[2 * x], s[2 * x + 1]);
            k2[x] = pack_bf16(s[32 + 2 * x], s[33 + 2 * x]);
          }
          tmem_st16_bits(tS + 16 * c, k1);       // over columns of S_1 that were read
          tmem_st16_bits(tS + 64 + 16 * c, k2);  // and of S_2
        }
        if (kMask && (words[0] & words[1]) != 0xffffffffu) {
          // K's rows outside the mask are read as zeros by the dQ product; S_1 and S_2 have been formed
          const int r = (threadIdx.x & 127) >> 1, half = threadIdx.x & 1;
          if (!((words[r >> 5] >> (r & 31)) & 1u)) {
            uint8_t* p = smem + L::kK + slot * L::kStepBytes + r * 128 + (D == 128 ? half * kStepChunk : half * 64);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) *reinterpret_cast<uint4*>(p + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&ctl->bar_ds_ready[wg]);
      }
      if (!ok) break;
      G0 += n;
      // epilogue: dQ = scale * (dS K)
      if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dq_done, it & 1, ctx, ctl)))) break;
      tc_fence_after();
      const uint32_t cQ = tl + kColDQ + 64 * wg + (D == 64 ? 32 * wg : 0);
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        float gv[32];
        tmem_ld32(cQ + 32 * c, gv);
        if (store) {
#pragma unroll
          for (int x = 0; x < 4; ++x) store8(dq + off + 32 * c + 8 * x, gv + 8 * x, scale);
        }
      }
      tc_fence_before();
      mbar_arrive(&ctl->bar_dq_free);
      ++it;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp && mma_issued) {
    mma_commit(&ctl->bar_final);
    settle(&ctl->bar_final, 0, ctx);
  }
  if (warp == kProducerWarp && lane == 0) {
    if (q_armed) settle(&ctl->bar_q_full, (q_armed - 1) & 1, ctx);
    for (int s = 0; s < R; ++s)
      if (armed[s]) settle(&ctl->bar_full[s], (armed[s] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename K>
int prepare(K kern, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess)
    return set_error(UAA_ERR_CUDA, "uaa_diff_attn_bwd: smem attribute: %s", cudaGetErrorString(e));
  return UAA_OK;
}

size_t row_floats(int B, int Sq, int H) { return (size_t)B * H * steps_of(Sq) * 4 * kStep; }

template <int D, bool kMask>
int launch_bwd(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const void* out,
               const void* out2, const void* dout, const float* lse, const uint8_t* mask, void* dq, void* dk, void* dv,
               void* dlam, int B, int Sq, int Sk, int H, float scale, float* rows, cudaStream_t s) {
  using bf = __nv_bfloat16;
  float* part = rows + row_floats(B, Sq, H);
  const int steps = steps_of(Sq);
  const long long items_k = (long long)tiles_of(Sk) * H * B, items_q = (long long)tiles_of(Sq) * H * B;
  const long long row_blocks = (long long)B * steps * ((H + kRowHeads - 1) / kRowHeads);
  if (items_k > INT32_MAX || items_q > INT32_MAX || row_blocks > INT32_MAX)
    return set_error(UAA_ERR_UNSUPPORTED, "uaa_diff_attn_bwd: too many work items");
  DevCtx ctx;
  SegMaps mq, mk, mv, mdo, sq, sk, sv, sdo;  // tiles of 128 rows, steps of 64
  const SeqDesc qd = seq_plain(Sq), kd = seq_plain(Sk);
  int st;
  if ((st = get_dev_ctx(&ctx)) || (st = encode_seq_maps(&mq, q, qd, B, H, D, kTile)) ||
      (st = encode_seq_maps(&mk, k, kd, B, H, D, kTile)) || (st = encode_seq_maps(&mv, v, kd, B, H, D, kTile)) ||
      (st = encode_seq_maps(&mdo, dout, qd, B, H, D, kTile)) || (st = encode_seq_maps(&sq, q, qd, B, H, D, kStep)) ||
      (st = encode_seq_maps(&sk, k, kd, B, H, D, kStep)) || (st = encode_seq_maps(&sv, v, kd, B, H, D, kStep)) ||
      (st = encode_seq_maps(&sdo, dout, qd, B, H, D, kStep)))
    return st;
  diff_rows_kernel<D><<<(int)row_blocks, kRowThreads, 0, s>>>(static_cast<const bf*>(out), static_cast<const bf*>(out2),
                                                             static_cast<const bf*>(dout), lse, lam, lam_bf16, rows,
                                                             part, B, Sq, H);
  if ((st = check_launch("uaa_diff_attn_bwd (rows)"))) return st;
  diff_dlambda_kernel<<<H, 256, 0, s>>>(part, dlam, lam_bf16, B * steps);
  if ((st = check_launch("uaa_diff_attn_bwd (dlambda)"))) return st;
  const int sms = device_sms();
  if (items_k > 0) {
    auto kern = diff_dkdv_kernel<D, kMask>;
    if ((st = prepare(kern, DkdvLayout<D>::kSmem))) return st;
    // with a key mask the heads go innermost while one batch's Q and dO fit in half of L2, so that the empty key
    // tiles spread evenly over the CTAs (as in the plain backward)
    const int head_inner = mask != nullptr && 4LL * H * Sq * D <= (64LL << 20);
    kern<<<(int)(items_k < sms ? items_k : sms), kThreads, DkdvLayout<D>::kSmem, s>>>(
        sq.m[0], mk.m[0], mv.m[0], sdo.m[0], lam, lam_bf16, rows, mask, static_cast<bf*>(dk), static_cast<bf*>(dv), B,
        H, Sq, Sk, (int)items_k, head_inner, scale, scale * kLog2e, ctx);
    if ((st = check_launch("uaa_diff_attn_bwd (dK/dV)"))) return st;
  }
  auto kern = diff_dq_kernel<D, kMask>;
  if ((st = prepare(kern, DqLayout<D>::kSmem))) return st;
  kern<<<(int)(items_q < sms ? items_q : sms), kThreads, DqLayout<D>::kSmem, s>>>(
      mq.m[0], sk.m[0], sv.m[0], mdo.m[0], lam, lam_bf16, rows, mask, static_cast<bf*>(dq), B, H, Sq, Sk, (int)items_q,
      scale, scale * kLog2e, ctx);
  return check_launch("uaa_diff_attn_bwd (dQ)");
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" size_t uaa_diff_attn_bwd_workspace_bytes(int B, int Sq, int H, int D) {
  if (B < 0 || Sq < 0 || H < 0 || (D != 64 && D != 128)) return 0;
  // the row vectors, and the sums of 64 rows' Delta_2
  return ((row_floats(B, Sq, H) + (size_t)B * H * steps_of(Sq)) * 4 + 255) & ~(size_t)255;
}

extern "C" int uaa_diff_attn_bwd(const void* q, const void* k, const void* v, const void* lambda, int lambda_dtype,
                                 const void* out, const void* out2, const void* dout, const float* lse,
                                 const uint8_t* key_mask, void* dq, void* dk, void* dv, void* dlambda, int B, int Sq,
                                 int Sk, int H, int D, float scale, void* workspace, size_t workspace_bytes,
                                 uaa_stream_t stream) {
  const char* fn = "uaa_diff_attn_bwd";
  int st = validate_attn_sizes(fn, B, Sq, Sk, H, D, scale);
  if (st) return st;
  if ((uint64_t)B * H == 0 || (uint64_t)Sq + Sk == 0) return UAA_OK;
  if (Sq == 0) return set_error(UAA_ERR_INVALID_ARG, "%s: keys without queries (Sq = 0)", fn);
  if ((st = check_dev_ptr(fn, "q", q)) || (st = check_dev_ptr(fn, "k", k)) || (st = check_dev_ptr(fn, "v", v)) ||
      (st = check_dev_ptr(fn, "out", out)) || (st = check_dev_ptr(fn, "out2", out2)) ||
      (st = check_dev_ptr(fn, "dout", dout)) || (st = check_dev_ptr(fn, "dq", dq)) ||
      (st = check_dev_ptr(fn, "dk", dk)) || (st = check_dev_ptr(fn, "dv", dv)) ||
      (st = check_lambda(fn, lambda, lambda_dtype)) || (st = check_lambda(fn, dlambda, lambda_dtype)) ||
      (st = check_lse(fn, lse)))
    return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  const size_t need = uaa_diff_attn_bwd_workspace_bytes(B, Sq, H, D);
  if (workspace_bytes < need)
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  auto go = D == 64 ? (key_mask ? launch_bwd<64, true> : launch_bwd<64, false>)
                    : (key_mask ? launch_bwd<128, true> : launch_bwd<128, false>);
  return go(q, k, v, lambda, lambda_dtype == UAA_BF16, out, out2, dout, lse, key_mask, dq, dk, dv, dlambda, B, Sq, Sk,
            H, scale, static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
}
