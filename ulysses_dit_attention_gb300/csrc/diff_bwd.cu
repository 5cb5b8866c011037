// Differential attention, backward (the formulas stand in diff_shared.cuh).
// No atomics: two runs on the same inputs give the same bits.
//  1. diff_rows_kernel: Delta_m and -LSE_m log2(e) of every query row, and the
//     sum of Delta_2 over 64 rows, the summands of dlambda.
//  2. diff_dkdv_kernel, key-tile-major: dK and dV of 128 keys.
//  3. diff_dq_kernel, query-tile-major: dQ of 128 queries; its loading warps, when they have loaded all and the
//     dK/dV kernel has ended, add up dlambda, in a fixed order.
// -lambda enters as |lambda| = 2^(log2 |lambda|), added to map 2's exponents with its LSE, and a sign: the negated
// A operand of map 2's dV product, and the sign of dQ_2 and dK_2 when they are written.
// Both matrix kernels: warps 0-15 compute (TMEM lane quadrant = warp % 4, 32 of a tile's 128 columns = warp / 4;
// four warps on each scheduler, because with two the latencies of TMEM and barriers lay open: dK/dV 1640 -> 1455 us,
// dQ 1067 -> 933 us at S = 8191, H = 24, D = 128), warp 16 loads by TMA, warp 17 issues the tcgen05 products from one
// elected lane.  MMAs of one thread run in order; two that read A from TMEM for different products are only relied on
// with equal shapes or with another product between them.
// At that size: 29 us, 1435 us (tensor pipe active 78 % of the time) and 862 us (66 %); 2.32 ms together.  What bounds the
// matrix kernels is the chain S -> P -> dS -> next S through TMEM and barriers, which one tile's products and the
// compute warps take in turns; two tiles half a step apart would need 640 columns of TMEM.
#include <algorithm>

#include "diff_shared.cuh"

namespace uaa {
namespace {

constexpr int kThreads = 576;
constexpr int kCompute = 512;  // warps 0-15
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
// Named barriers between the compute warps (which arrive) and the issuer (which syncs): the issuer waits on these
// within an item, because an mbarrier test would be held behind the MMAs that it has queued.
constexpr uint32_t kBarP = 1, kBarDS = 2, kBarCount = kCompute + 32;
constexpr uint32_t kBarSum = 3;  // the compute warps of the dK/dV kernel exchange their sums of dS_2
constexpr int kRowBytes = 4 * kTile * 4;
constexpr uint32_t kIdescNegateA = 1u << 13;  // instruction descriptor: the A operand is negated

// Row vectors, (B, H, tiles, 4, 128): -LSE_1 log2(e), -LSE_2 log2(e) + log2 |lambda|, Delta_1, Delta_2 of a tile's
// queries
__host__ __device__ __forceinline__ size_t row_floats(int B, int Sq, int H) {
  return (size_t)B * H * tiles_of(Sq) * 4 * kTile;
}
__host__ __device__ __forceinline__ size_t rows_at(size_t bh, int Sq, int i) {
  return (bh * tiles_of(Sq) + i / kTile) * (4 * kTile) + i % kTile;
}

// TMEM column of the A operand for 16-element step kk: each warpgroup's 32 packed elements lie in the first 16
// columns of its own 32.
__device__ __forceinline__ uint32_t packed_col(int kk) { return 32 * (kk >> 1) + 8 * (kk & 1); }

// 32 values as bf16 pairs into 16 columns of this thread's TMEM lane, then a wait for the store.
__device__ __forceinline__ void store_packed32(uint32_t taddr, const float (&x)[32]) {
  uint32_t v[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
  tmem_st16_bits(taddr, v);
}

// Are these barriers' phases complete?  Both are tested before either answer is used; the slow path waits in turn.
template <typename Ctl>
__device__ __forceinline__ bool wait_two(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, const DevCtx& ctx,
                                         Ctl* ctl) {
  dbg_late(ctx);
  const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
  if (ra && rb) return true;
  return wait_or_abort(a, pa, ctx, ctl) && wait_or_abort(b, pb, ctx, ctl);
}

// Pieces of 16 bytes, N of this lane's row, to piece lane % N of the N rows of its group of N lanes: a store of the warp
// then writes 32 / N rows, 16 N bytes each, instead of 16 bytes in each of 32 rows.
template <int N>
__device__ __forceinline__ void swap_pieces(uint4 (&x)[N], int lane) {
#pragma unroll
  for (int bit = 1; bit < N; bit *= 2) {
    const bool hi = lane & bit;
#pragma unroll
    for (int p = 0; p < N; ++p) {
      if (p & bit) continue;
      uint4 v = hi ? x[p] : x[p | bit];
      v.x = __shfl_xor_sync(0xffffffffu, v.x, bit), v.y = __shfl_xor_sync(0xffffffffu, v.y, bit);
      v.z = __shfl_xor_sync(0xffffffffu, v.z, bit), v.w = __shfl_xor_sync(0xffffffffu, v.w, bit);
      (hi ? x[p] : x[p | bit]) = v;
    }
  }
}

// Warp-collective: 8 N accumulator columns of 32 rows, times c (zero where `zero`), as bf16; row 0 of them at `at`, the
// rows `pitch` elements apart, `left` of them to be written.
template <int N>
__device__ __forceinline__ void store_rows(__nv_bfloat16* base, size_t at, size_t pitch, int left, uint32_t col, float c,
                                           bool zero, int lane, const DevCtx& ctx, size_t extent) {
  uint4 x[N];
#pragma unroll
  for (int h = 0; h < N / 2; ++h) {
    float v[16];
    tmem_ld16(col + 16 * h, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = zero ? 0.f : v[i] * c;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x[2 * h + i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
  }
  swap_pieces<N>(x, lane);
  const int q = lane % N, r0 = lane - q;
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const size_t to = at + (r0 + r) * pitch + 8 * q;
    if (r0 + r < left && guard_store(ctx, to, 8, extent)) *reinterpret_cast<uint4*>(base + to) = x[r];
  }
}

// ---------------------------------------------------------------------------
// 1. Row vectors.  Bound: reading O, O2 and dO once.  A block takes 64 rows of one head, D/8 lanes of 16 bytes a row
// and all of a lane's rows in flight; neighbouring blocks take neighbouring heads, whose rows lie side by side.
// 29 us at B = 1, S = 8191, H = 24, D = 128 (5.3 TB/s; four heads a block one after the other: 47 us).
constexpr int kRowThreads = 256;
constexpr int kStep = 64;
__host__ __device__ __forceinline__ int steps_of(int S) { return 2 * tiles_of(S); }

// The three kernels of a call overlap at their ends (programmatic dependent launch): when all blocks of a kernel have
// called allow_next(), the next one's start wherever an SM has room; await_previous() returns when the previous kernel
// has completed and its writes can be read.  The dK/dV kernel waits for the row vectors before it lets the dQ kernel
// start, and the dQ kernel, which needs nothing of the dK/dV kernel's but sums for dlambda and reads the row kernel's
// values past L1, waits for it at its end, so that a call is complete when its last kernel is.  One launch after the
// other against this: 69.6 -> 56.8 us at B = 2, S = 1000, H = 12, D = 64; 807 -> 775 us at B = 2, S = 4096, H = 24,
// D = 128 with a mask; 2473 -> 2405 us at S = 8191, H = 24, D = 128.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kRowThreads) diff_rows_kernel(
    const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ out2,
    const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse, const void* __restrict__ lam, int lam_bf16,
    float* __restrict__ rows, float* __restrict__ part, int B, int Sq, int H, DevCtx ctx) {
  constexpr int G = D / 8;
  constexpr int kGroups = kRowThreads / G;
  __shared__ float sums[kGroups];
  allow_next();
  const int group = threadIdx.x / G, sub = threadIdx.x % G;
  const int steps = steps_of(Sq);
  const int h = blockIdx.x % H, t = blockIdx.x / H % steps, b = blockIdx.x / H / steps;
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
        // rows past Sq, or without a key: P = 0; where a score was NaN or +inf (LSE = NaN or +inf): P = NaN
        x = l == -INFINITY ? -INFINITY : l < INFINITY ? -l * kLog2e : NAN;
        if (sub == 1 && l != -INFINITY) x += log2f(fabsf(lm));
      }
      const size_t to = rows_at(bh, Sq, i) + sub * kTile;
      if (guard_store(ctx, to, 1, row_floats(B, Sq, H))) rows[to] = x;
    }
  }
  if (sub == 0) sums[group] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int x = 0; x < kGroups; ++x) s += sums[x];
    const size_t to = (size_t)h * B * steps + (size_t)b * steps + t;
    if (guard_store(ctx, to, 1, (size_t)B * H * steps)) part[to] = s;
  }
}

// dlambda_h = -sum of Delta_2 over the head's rows, by one warp, in a fixed order.  The row kernel's Delta_2 (part) holds
// the rounding of O_2 to bf16, which the sum, often small against its summands, would show: 0.4 % and more.  But
// sum_j dS_2 of a row is -lambda (Delta_2 - that value), as A_2 sums to 1, so the dK/dV kernel, which has dS_2 in 32
// bits, leaves what is missing in its items' sums (rest).
__device__ __forceinline__ void sum_dlambda(const float* part, int n, const float* rest, int n_rest,
                                            void* __restrict__ dlam, int lam_bf16, int h, int lane) {
  float s = 0.f;
#pragma unroll 4
  for (int i = lane; i < n; i += 32) s += __ldcg(part + (size_t)h * n + i);
#pragma unroll 4
  for (int i = lane; i < n_rest; i += 32) s += __ldcg(rest + (size_t)h * n_rest + i);
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
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
// 2. dK, dV.  A persistent CTA takes 128 keys of one (batch, head); its steps are the maps of the query tiles in
// turn, (i, 1) (i, 2) (i + 1, 1) ...:
//     S^T = K_m Q_m^T, P^T = w_m A_m^T (w = 1, -lambda), dA^T = V dO^T    (M = keys, N = 128 queries)
//     dV += P^T dO, dS^T = P^T (dA^T - Delta_m), dK_m += dS^T Q_m
// One elected lane issues, per step: dV_s S_{s+1} after P_s, dK_s dA_{s+1} after dS_s; so the tensor cores work
// while the compute warps take the exponentials of the next step or form dS of this one.  dA is formed anew for the
// second map.  Kept in the compute warps' registers instead, it saves a seventh of the MMAs and no time: 2401 against
// 2343 us for the whole backward at B = 1, S = 8191, H = 24, D = 128, 773 against 750 at B = 2, S = 4096 with a mask;
// nor does one dV product of A_1 - lambda A_2 (2727).  Steps of 64 queries, whose TMEM would hold two buffers, lose
// too: a product with both operands in shared memory takes as long for 64 columns as for 128 (2052 against 1640 us,
// with eight compute warps).
// TMEM: S^T at column 0, dA^T at 128 (P^T and dS^T, packed, over the first 16 columns of each warpgroup's 32),
// dV at 256, dK_m at 384 + 64 m (with D = 64 the product runs over all 64 columns of Q and map m's 32 are kept).
template <int D>
struct DkdvLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kRing = D == 128 ? 2 : 4;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQ = kV + kTileBytes;
  static constexpr int kDO = kQ + kRing * kTileBytes;
  static constexpr int kRows = kDO + kRing * kTileBytes;
  static constexpr int kCtl = kRows + kRing * kRowBytes;
  static constexpr int kSmem = kCtl + 256;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

struct DkdvCtl {
  uint64_t bar_kv_full, bar_kv_empty;
  uint64_t bar_full[4], bar_empty[4];
  uint64_t bar_s_full, bar_dp_full, bar_dv_done;
  uint64_t bar_acc_done, bar_acc_free, bar_final;
  uint32_t tmem_base;
  int abort;
  float sums[16];  // a warp's sum of dS_2 over an item
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
                     __nv_bfloat16* __restrict__ dv, float* __restrict__ rest, int B, int H, int Sq, int Sk,
                     int num_items, int head_inner,
                     float scale, float scale_log2, DevCtx ctx) {
  using L = DkdvLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, kTile, false, false);  // S^T, dA^T
  constexpr uint32_t kIdescV = idesc_bf16_f32(128, D, false, true);       // dV (A in TMEM)
  constexpr uint32_t kIdescK = idesc_bf16_f32(128, 64, false, true);      // dK_m (A in TMEM)
  constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 384;

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
  const int nqt = tiles_of(Sq);

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_kv_full, 1);
    mbar_init(&ctl->bar_kv_empty, 1);
    for (int s = 0; s < R; ++s) {
      mbar_init(&ctl->bar_full[s], 1);
      mbar_init(&ctl->bar_empty[s], 1);
    }
    mbar_init(&ctl->bar_s_full, 1);
    mbar_init(&ctl->bar_dp_full, 1);
    mbar_init(&ctl->bar_dv_done, 1);
    mbar_init(&ctl->bar_acc_done, 1);
    mbar_init(&ctl->bar_acc_free, kCompute);
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
  await_previous();  // the row vectors
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  allow_next();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t k_extent = (size_t)B * Sk * H * D;

  uint32_t armed[4] = {}, kv_armed = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t T = 0, it = 0;  // query tiles and items so far
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
        for (int i = 0; ok && i < nqt; ++i, ++T) {
          const int slot = T % R;
          const uint32_t use = T / R;
          if (use > 0) ok = wait_or_abort(&ctl->bar_empty[slot], (use - 1) & 1, ctx, ctl);
          if (!ok) break;
          if ((int)T == ctx.drop_load) continue;
          mbar_arrive_expect_tx(&ctl->bar_full[slot], 2 * L::kTileBytes + kRowBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kQ + slot * L::kTileBytes + c * kChunkBytes, &tmQ, &ctl->bar_full[slot], c * 64, w.h,
                        i * kTile, w.b);
            tma_load_4d(smem + L::kDO + slot * L::kTileBytes + c * kChunkBytes, &tmDO, &ctl->bar_full[slot], c * 64,
                        w.h, i * kTile, w.b);
          }
          bulk_load(smem + L::kRows + slot * kRowBytes, rsrc + (size_t)i * 4 * kTile, kRowBytes, &ctl->bar_full[slot]);
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
    uint32_t T0 = 0, it = 0;
    auto wait_el = [&](uint64_t* bar, uint32_t parity) {
      bool w = true;
      if (el) w = wait_or_abort(bar, parity, ctx, ctl);
      return __shfl_sync(0xffffffffu, w ? 1 : 0, el_lane) != 0;
    };
    auto sq = [&](uint32_t T) { return sbase + L::kQ + (T % R) * L::kTileBytes; };
    auto sdo = [&](uint32_t T) { return sbase + L::kDO + (T % R) * L::kTileBytes; };
    auto issue_s = [&](uint32_t T, int m) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kK, 16, 1024), b0 = sdesc_sw128(sq(T), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const uint32_t off = m ? map_step<D>(1, kk) : map_step<D>(0, kk);
        const uint64_t a = desc_add(a0, off), b = desc_add(b0, off);
        if (el) mma_ss_checked(mg, tmem + kColS, a, b, kIdescS, kk > 0, kTile);
      }
      if (el) mma_commit(&ctl->bar_s_full);
    };
    auto issue_dp = [&](uint32_t T) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kV, 16, 1024), b0 = sdesc_sw128(sdo(T), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
        const uint64_t a = desc_add(a0, off), b = desc_add(b0, off);
        if (el) mma_ss_checked(mg, tmem + kColDP, a, b, kIdescS, kk > 0, kTile);
      }
      if (el) mma_commit(&ctl->bar_dp_full);
    };
    auto issue_dv = [&](uint32_t T, bool first, bool last, uint32_t idesc) {
      const uint64_t b0 = sdesc_sw128(sdo(T), kChunkBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint64_t b = desc_add(b0, kk * 2048);
        if (el)
          mma_ts_checked(mg, tmem + kColDV, tmem + kColS + packed_col(kk), b, idesc, (!first || kk > 0) ? 1u : 0u, D);
      }
      if (el && last) mma_commit(&ctl->bar_dv_done);
    };
    auto issue_dk = [&](uint32_t T, int m, bool first) {
      const uint64_t b0 = sdesc_sw128(sq(T) + (D == 128 ? m * kChunkBytes : 0), kChunkBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint64_t b = desc_add(b0, kk * 2048);
        if (el)
          mma_ts_checked(mg, tmem + kColDK + 64 * m, tmem + kColDP + packed_col(kk), b, kIdescK,
                         (!first || kk > 0) ? 1u : 0u, 64);
      }
      if (el && m == 1) mma_commit(&ctl->bar_empty[T % R]);
    };
    for (int item = blockIdx.x; item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nkt, H, head_inner);
      if (kMask && !tile_any(key_mask, w.b, w.t, Sk)) continue;
      // After a failure anywhere in the CTA this warp stops issuing but still meets the compute warps at
      // every named barrier of the schedule.
      if (ok && *reinterpret_cast<volatile int*>(&ctl->abort)) ok = false;
      // map 2's probabilities enter dV with the sign of -lambda
      const uint32_t idesc2 = kIdescV | (load_lambda(lam, lam_bf16, w.h) > 0.f ? kIdescNegateA : 0u);
      if (ok) ok = wait_el(&ctl->bar_kv_full, it & 1);
      if (ok) ok = wait_el(&ctl->bar_full[T0 % R], (T0 / R) & 1);
      if (ok) {
        tc_fence_after();
        issue_s(T0, 0);
        issue_dp(T0);
        if (el) mma_issued = true;
      }
      for (int i = 0; i < nqt; ++i) {
        const uint32_t T = T0 + i;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const bool more = m == 0 || i + 1 < nqt;
          const uint32_t T1 = T + m;  // the next step's tile
          // P is in TMEM, and the next step's Q has landed: the compute warps waited for it
          named_sync(kBarP, kBarCount);
          // the previous item's epilogue must have read dV and dK
          if (ok && i == 0 && m == 0 && it > 0) ok = wait_el(&ctl->bar_acc_free, (it - 1) & 1);
          if (ok) {
            tc_fence_after();
            issue_dv(T, i == 0 && m == 0, !more, m ? idesc2 : kIdescV);
            if (more) issue_s(T1, 1 - m);
          }
          __syncwarp();
          named_sync(kBarDS, kBarCount);
          if (ok) {
            tc_fence_after();
            issue_dk(T, m, i == 0);
            if (more) issue_dp(T1);
          }
          __syncwarp();
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
      T0 += nqt;
      ++it;
    }
  } else {
    // ------------------------------------------------------------ compute: quarter cq of the queries of every step
    const int cq = warp >> 2;
    const int jrow = (warp & 3) * 32 + lane;  // key row = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + kColS + 32 * cq, tP = tl + kColDP + 32 * cq;
    bool ok = true;
    uint32_t T0 = 0, G = 0, it = 0;  // G: steps so far
    for (int item = blockIdx.x; item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nkt, H, head_inner);
      const int j = w.t * kTile + jrow;
      const bool exists = j < Sk;
      // this thread writes a quarter of the row's columns
      const size_t off = (((size_t)w.b * Sk + (exists ? j : 0)) * H + w.h) * D + cq * (D / 4);
      const bool store = exists && guard_store(ctx, off, D / 4, k_extent);
      const size_t rest_at = ((size_t)w.h * B + w.b) * nkt + w.t;
      const bool rest_store = threadIdx.x == 0 && guard_store(ctx, rest_at, 1, (size_t)B * H * nkt);
      if (kMask && !tile_any(key_mask, w.b, w.t, Sk)) {
        // no attended key in this tile: dK = dV = 0
        if (rest_store) rest[rest_at] = 0.f;
        if (store) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            *reinterpret_cast<uint4*>(dk + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(dv + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      const float2 c2 = make_float2(scale_log2, scale_log2);
      float2 sum = make_float2(0.f, 0.f);  // of this key's dS_2, with |lambda|
      for (int i = 0; i < nqt; ++i) {
        const uint32_t T = T0 + i, slot = T % R;
        const bool last = i + 1 == nqt;
#pragma unroll
        for (int m = 0; m < 2; ++m, ++G) {
          const float* rv = reinterpret_cast<const float*>(smem + L::kRows + slot * kRowBytes) + m * kTile + 32 * cq;
          if (ok) {
            // S, and the row vectors with this tile (m = 0), or the next tile, which the product released by this
            // step's first arrival reads
            const uint32_t Tw = m == 0 || last ? T : T + 1;
            ok = __all_sync(0xffffffffu, wait_two(&ctl->bar_s_full, G & 1, &ctl->bar_full[Tw % R], (Tw / R) & 1, ctx,
                                                  ctl));
          }
          if (!ok) {
            // after a failure: keep meeting the issuer, a rendezvous at every step of the schedule
            named_sync(kBarP, kBarCount);
            named_sync(kBarDS, kBarCount);
            continue;
          }
          tc_fence_after();
          float p[32];  // A_1 or |lambda| A_2
          tmem_ld32(tS, p);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 r = *reinterpret_cast<const float4*>(rv + 4 * c);
            const float2 x = fma2(make_float2(p[4 * c], p[4 * c + 1]), c2, make_float2(r.x, r.y));
            const float2 y = fma2(make_float2(p[4 * c + 2], p[4 * c + 3]), c2, make_float2(r.z, r.w));
            p[4 * c] = ex2(x.x), p[4 * c + 1] = ex2(x.y), p[4 * c + 2] = ex2(y.x), p[4 * c + 3] = ex2(y.y);
          }
          store_packed32(tS, p);
          tc_fence_before();
          named_arrive(kBarP, kBarCount);
          ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dp_full, G & 1, ctx, ctl));
          if (!ok) {
            named_sync(kBarDS, kBarCount);
            continue;
          }
          tc_fence_after();
          float dp[32];
          tmem_ld32(tP, dp);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 r = *reinterpret_cast<const float4*>(rv + 2 * kTile + 4 * c);
            const float2 x = mul2(make_float2(p[4 * c], p[4 * c + 1]),
                                  sub2(make_float2(dp[4 * c], dp[4 * c + 1]), make_float2(r.x, r.y)));
            const float2 y = mul2(make_float2(p[4 * c + 2], p[4 * c + 3]),
                                  sub2(make_float2(dp[4 * c + 2], dp[4 * c + 3]), make_float2(r.z, r.w)));
            dp[4 * c] = x.x, dp[4 * c + 1] = x.y, dp[4 * c + 2] = y.x, dp[4 * c + 3] = y.y;
          }
          store_packed32(tP, dp);
          // dV's and dK's products both read A from TMEM and differ in shape: where no other product stands
          // between them, dV has to have completed
          if (m == 1 && last) ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dv_done, it & 1, ctx, ctl));
          tc_fence_before();
          named_arrive(kBarDS, kBarCount);
          if (m == 1) {
#pragma unroll
            for (int c = 0; c < 16; ++c) sum = add2(sum, make_float2(dp[2 * c], dp[2 * c + 1]));
          }
        }
      }
      T0 += nqt;
      const bool attended = exists && (!kMask || key_mask[(size_t)w.b * Sk + j] != 0);
      float total = attended ? sum.x + sum.y : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) total += __shfl_xor_sync(0xffffffffu, total, o);
      if (lane == 0) ctl->sums[warp] = total;
      named_sync(kBarSum, kCompute);
      if (rest_store) {
        // where lambda is 0, or so small that dS_2 may be, the row kernel's sum stands
        const float l = fabsf(load_lambda(lam, lam_bf16, w.h));
        total = 0.f;
        for (int x = 0; x < kCompute / 32; ++x) total += ctl->sums[x];
        rest[rest_at] = l >= 0x1p-60f ? total / l : 0.f;
      }
      // epilogue: dV, and dK = scale * (dS^T Q).  A key outside the mask gets zeros, whatever its rows hold.
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_acc_done, it & 1, ctx, ctl));
      ++it;
      if (!ok) continue;
      tc_fence_after();
      const float ck = cq >= 2 && load_lambda(lam, lam_bf16, w.h) > 0.f ? -scale : scale;
      const uint32_t cV = tl + kColDV + cq * (D / 4);
      const uint32_t cK = tl + kColDK + cq * (D / 4) + (D == 64 ? (cq >> 1) * 64 : 0);
      const int j0 = w.t * kTile + (warp & 3) * 32;
      const size_t to = (((size_t)w.b * Sk + j0) * H + w.h) * D + cq * (D / 4), pitch = (size_t)H * D;
      store_rows<D / 32>(dv, to, pitch, Sk - j0, cV, 1.f, !attended, lane, ctx, k_extent);
      store_rows<D / 32>(dk, to, pitch, Sk - j0, cK, ck, !attended, lane, ctx, k_extent);
      tc_fence_before();
      mbar_arrive(&ctl->bar_acc_free);
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
// 3. dQ.  A persistent CTA takes 128 queries of one (batch, head), Q and dO in shared memory, and walks the key
// tiles: S_m = Q_m K_m^T, dA = dO V^T (M = queries, N = 128 keys), then dQ_m += dS_m K_m.  The maps take turns:
// while the compute warps work on map 2 of tile g, with dA in their registers, the tensor cores form dQ_1 of tile g, S_1
// and dA of tile g + 1; then dQ_2 and S_2 while they take map 1's exponentials.
// TMEM: S_1 at column 0, S_2 at 128 (dS_m, packed, over the first 16 columns of each warpgroup's 32), dA at 256,
// dQ_m at 384 + 64 m (with D = 64 the product runs over all 64 columns of K and map m's 32 are kept).
template <int D>
struct DqLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kKRing = D == 128 ? 3 : 6;  // a K slot is freed by dQ_2, a V slot already by dA
  static constexpr int kVRing = D == 128 ? 2 : 5;
  static constexpr int kQ = 0;
  static constexpr int kDO = kQ + kTileBytes;
  static constexpr int kK = kDO + kTileBytes;
  static constexpr int kV = kK + kKRing * kTileBytes;
  static constexpr int kCtl = kV + kVRing * kTileBytes;
  static constexpr int kCnt = kCtl + 384;  // attended key tiles per mask row
  static constexpr int kSmem = kCnt + kMaxCntRows * 4;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

// The items of a CTA: one of every `all` rounds over the whole grid, then, for the first `early` CTAs, one of every
// further round over these.  The first CTAs start on SMs that the dK/dV kernel's last round leaves idle.
struct DqWalk {
  int all, early;
};
__device__ __forceinline__ int next_item(const DqWalk& w, int item, int num_items) {
  const int grid = gridDim.x, head = min(w.all, num_items / grid + 1) * grid;  // the items of the first rounds
  if (item + grid < head) return item + grid;
  if ((int)blockIdx.x >= w.early) return num_items;
  return item < head ? head + (int)blockIdx.x : item + w.early;
}

struct DqCtl {
  uint64_t bar_q_full, bar_q_empty;
  uint64_t bar_k_full[6], bar_k_empty[6], bar_v_full[5], bar_v_empty[5];
  uint64_t bar_s_full[2], bar_dp_full;
  uint64_t bar_dq_done, bar_dq_free, bar_final;
  uint32_t tmem_base;
  int abort;
  uint32_t mask_words[6][4];  // per K slot: the attended keys of its tile
};
static_assert(sizeof(DqCtl) <= 384, "control block");

template <int D, bool kMask>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                   const void* __restrict__ lam, int lam_bf16, const float* __restrict__ rows,
                   const uint8_t* __restrict__ key_mask, __nv_bfloat16* __restrict__ dq,
                   const float* part, const float* rest, void* __restrict__ dlam, int B, int H, int Sq, int Sk,
                   int num_items, DqWalk walk, float scale, float scale_log2, DevCtx ctx) {
  using L = DqLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int KR = L::kKRing, VR = L::kVRing;
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, kTile, false, false);  // S, dA
  constexpr uint32_t kIdescQ = idesc_bf16_f32(128, 64, false, true);      // dQ_m (A in TMEM)
  constexpr uint32_t kColDP = 256, kColDQ = 384;

  extern __shared__ __align__(1024) uint8_t smem[];
  DqCtl* ctl = reinterpret_cast<DqCtl*>(smem + L::kCtl);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    await_previous();
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nqt = tiles_of(Sq);
  const int nkt = tiles_of(Sk);

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_q_full, 1);
    mbar_init(&ctl->bar_q_empty, 1);
    for (int s = 0; s < KR; ++s) {
      mbar_init(&ctl->bar_k_full[s], 1);
      mbar_init(&ctl->bar_k_empty[s], 1);
    }
    for (int s = 0; s < VR; ++s) {
      mbar_init(&ctl->bar_v_full[s], 1);
      mbar_init(&ctl->bar_v_empty[s], 1);
    }
    mbar_init(&ctl->bar_s_full[0], 1);
    mbar_init(&ctl->bar_s_full[1], 1);
    mbar_init(&ctl->bar_dp_full, 1);
    mbar_init(&ctl->bar_dq_done, 1);
    mbar_init(&ctl->bar_dq_free, kCompute);
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
  // Attended key tiles per mask row: every role takes its tile count from this table, which no one writes after the
  // start; only the producer reads the mask itself and leaves each tile's bits with its K slot.
  int* tile_cnt = reinterpret_cast<int*>(smem + L::kCnt);
  const bool skip = kMask && B <= kMaxCntRows;
  if (skip) {
    for (int r = threadIdx.x; r < B; r += kThreads) tile_cnt[r] = 0;
    __syncthreads();
    for (int pr = warp; pr < B * nkt; pr += kThreads / 32)
      if (tile_any(key_mask, pr / nkt, pr % nkt, Sk) && lane == 0) atomicAdd(&tile_cnt[pr / nkt], 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t q_extent = (size_t)B * Sq * H * D;
  auto item_tiles = [&](int b) { return skip ? tile_cnt[b] : nkt; };

  uint32_t k_armed[6] = {}, v_armed[5] = {}, q_armed = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t G = 0, it = 0;
    for (int item = blockIdx.x; ok && item < num_items; item = next_item(walk, item, num_items)) {
      const Item w = decode_item(item, nqt, H, false);
      if (item_tiles(w.b) == 0) continue;  // no attended key: the compute warps write dQ = 0
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
      for (int j = 0; ok && j < nkt; ++j) {
        uint32_t words[4] = {0u, 0u, 0u, 0u};
        if (kMask) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int c = j * kTile + 32 * t + lane;
            words[t] = __ballot_sync(0xffffffffu, c < Sk && key_mask[(size_t)w.b * Sk + c] != 0);
          }
          if (skip && (words[0] | words[1] | words[2] | words[3]) == 0) continue;
        }
        if (lane == 0) {
          const int ks = G % KR, vs = G % VR;
          if (G / KR > 0) ok = wait_or_abort(&ctl->bar_k_empty[ks], (G / KR - 1) & 1, ctx, ctl);
          if (ok) {
#pragma unroll
            for (int t = 0; t < 4; ++t) ctl->mask_words[ks][t] = words[t];
            if ((int)G != ctx.drop_load) {
              mbar_arrive_expect_tx(&ctl->bar_k_full[ks], L::kTileBytes);
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(smem + L::kK + ks * L::kTileBytes + c * kChunkBytes, &tmK, &ctl->bar_k_full[ks], c * 64,
                            w.h, j * kTile, w.b);
              k_armed[ks] = G / KR + 1;
            }
            if (G / VR > 0) ok = wait_or_abort(&ctl->bar_v_empty[vs], (G / VR - 1) & 1, ctx, ctl);
          }
          if (ok) {
            mbar_arrive_expect_tx(&ctl->bar_v_full[vs], L::kTileBytes);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(smem + L::kV + vs * L::kTileBytes + c * kChunkBytes, &tmV, &ctl->bar_v_full[vs], c * 64, w.h,
                          j * kTile, w.b);
            v_armed[vs] = G / VR + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++G;
      }
    }
    if (blockIdx.x < H) await_previous();  // the sums of the dK/dV kernel
    for (int h = blockIdx.x; h < H; h += gridDim.x)
      sum_dlambda(part, B * steps_of(Sq), rest, B * nkt, dlam, lam_bf16, h, lane);
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
    auto sk = [&](uint32_t G) { return sbase + L::kK + (G % KR) * L::kTileBytes; };
    auto issue_s = [&](uint32_t G, int m) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kQ, 16, 1024), b0 = sdesc_sw128(sk(G), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const uint32_t off = m ? map_step<D>(1, kk) : map_step<D>(0, kk);
        const uint64_t a = desc_add(a0, off), b = desc_add(b0, off);
        if (el) mma_ss_checked(mg, tmem + m * kTile, a, b, kIdescS, kk > 0, kTile);
      }
      if (el) mma_commit(&ctl->bar_s_full[m]);
    };
    auto issue_dp = [&](uint32_t G) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kDO, 16, 1024);
      const uint64_t b0 = sdesc_sw128(sbase + L::kV + (G % VR) * L::kTileBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
        const uint64_t a = desc_add(a0, off), b = desc_add(b0, off);
        if (el) mma_ss_checked(mg, tmem + kColDP, a, b, kIdescS, kk > 0, kTile);
      }
      if (el) {
        mma_commit(&ctl->bar_dp_full);
        mma_commit(&ctl->bar_v_empty[G % VR]);
      }
    };
    auto issue_dq = [&](uint32_t G, int m, bool first) {
      const uint64_t b0 = sdesc_sw128(sk(G) + (D == 128 ? m * kChunkBytes : 0), kChunkBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        const uint64_t b = desc_add(b0, kk * 2048);
        if (el)
          mma_ts_checked(mg, tmem + kColDQ + 64 * m, tmem + m * kTile + packed_col(kk), b, kIdescQ,
                         (!first || kk > 0) ? 1u : 0u, 64);
      }
      if (el && m == 1) mma_commit(&ctl->bar_k_empty[G % KR]);
    };
    for (int item = blockIdx.x; item < num_items; item = next_item(walk, item, num_items)) {
      const Item w = decode_item(item, nqt, H, false);
      const int n = item_tiles(w.b);
      if (n == 0) continue;
      if (ok && *reinterpret_cast<volatile int*>(&ctl->abort)) ok = false;  // see the dK/dV kernel
      if (ok) ok = wait_el(&ctl->bar_q_full, it & 1);
      if (ok) ok = wait_el(&ctl->bar_k_full[G0 % KR], (G0 / KR) & 1);
      if (ok) {
        tc_fence_after();
        issue_s(G0, 0);
        if (el) mma_issued = true;
        ok = wait_el(&ctl->bar_v_full[G0 % VR], (G0 / VR) & 1);
      }
      if (ok) {
        tc_fence_after();
        issue_dp(G0);
        issue_s(G0, 1);
        if (el && n == 1) mma_commit(&ctl->bar_q_empty);
      }
      for (int g = 0; g < n; ++g) {
        const uint32_t G = G0 + g;
        const bool more = g + 1 < n;
        // dS_1 is in TMEM, dA has been read, and the next K and V tiles have landed: the compute warps waited for them
        named_sync(kBarP, kBarCount);
        // the previous item's epilogue must have read dQ
        if (ok && g == 0 && it > 0) ok = wait_el(&ctl->bar_dq_free, (it - 1) & 1);
        if (ok) {
          tc_fence_after();
          issue_dq(G, 0, g == 0);
          if (more) {
            issue_s(G + 1, 0);
            issue_dp(G + 1);
          }
        }
        __syncwarp();
        // dS_2 is in TMEM
        named_sync(kBarDS, kBarCount);
        if (ok) {
          tc_fence_after();
          issue_dq(G, 1, g == 0);
          if (more) {
            issue_s(G + 1, 1);
            if (el && g + 2 == n) mma_commit(&ctl->bar_q_empty);  // the item's last products with Q and dO
          }
        }
        __syncwarp();
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
    // ------------------------------------------------------------ compute: quarter cq of the keys of every tile
    const int cq = warp >> 2;
    const int row = (warp & 3) * 32 + lane;  // query row = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + 32 * cq;
    bool ok = true;
    uint32_t G0 = 0, it = 0;
    for (int item = blockIdx.x; item < num_items; item = next_item(walk, item, num_items)) {
      const Item w = decode_item(item, nqt, H, false);
      const int n = item_tiles(w.b);
      const int i = w.t * kTile + row;
      // this thread writes a quarter of the row's columns
      const size_t off = (((size_t)w.b * Sq + (i < Sq ? i : 0)) * H + w.h) * D + cq * (D / 4);
      const bool store = i < Sq && guard_store(ctx, off, D / 4, q_extent);
      if (n == 0) {
        if (store) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) *reinterpret_cast<uint4*>(dq + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      const float* rv = rows + rows_at((size_t)w.b * H + w.h, Sq, i);  // rows past Sq: -inf and 0
      const float2 c2 = make_float2(scale_log2, scale_log2);
      const float nl2[2] = {__ldcg(rv), __ldcg(rv + kTile)}, delta[2] = {__ldcg(rv + 2 * kTile), __ldcg(rv + 3 * kTile)};
      for (int g = 0; g < n; ++g) {
        const uint32_t G = G0 + g, ks = G % KR;
        const bool more = g + 1 < n;
        if (ok) {
          // S_1, and the next K tile, which the product released by this tile's first arrival reads
          const uint32_t Gw = more ? G + 1 : G;
          ok = __all_sync(0xffffffffu, wait_two(&ctl->bar_s_full[0], G & 1, &ctl->bar_k_full[Gw % KR], (Gw / KR) & 1,
                                                ctx, ctl));
        }
        if (!ok) {
          // after a failure: keep meeting the issuer
          named_sync(kBarP, kBarCount);
          named_sync(kBarDS, kBarCount);
          continue;
        }
        uint32_t word = 0xffffffffu;  // the attended keys of this quarter
        if (kMask) {
          if (g == 0) ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_k_full[ks], (G / KR) & 1, ctx, ctl));
          word = ctl->mask_words[ks][cq];
          // K's rows outside the mask are read as zeros by the dQ products; where S_2 is still being formed, it
          // is only masked columns that change
          const int r = threadIdx.x >> 2;
          if (!((ctl->mask_words[ks][r >> 5] >> (r & 31)) & 1u)) {
            const int x = (threadIdx.x & 3) * (D / 2);  // byte of the row's 2 D, in 128-byte chunks
            uint8_t* z = smem + L::kK + ks * L::kTileBytes + (x >> 7) * kChunkBytes + r * 128 + (x & 127);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) *reinterpret_cast<uint4*>(z + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        } else if (!more) {  // keys past the end
          const int left = Sk - (nkt - 1) * kTile - 32 * cq;
          word = left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1u : 0u);
        }
        bool met = false;  // this tile's first arrival has been made
        float dp[32];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          if (m == 1) {
            met = true;
            ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_s_full[1], G & 1, ctx, ctl));
            if (!ok) break;
          }
          tc_fence_after();
          float p[32];  // A_1 or |lambda| A_2
          tmem_ld32(tS + m * kTile, p);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 x = fma2(make_float2(p[2 * c], p[2 * c + 1]), c2, make_float2(nl2[m], nl2[m]));
            p[2 * c] = ex2(x.x), p[2 * c + 1] = ex2(x.y);
          }
          if (m == 0) {
            // dA, and the next V tile, which the next dA's product reads as soon as this one has been read.  Behind an
            // item's last tile that is the next item's, and the issuer waits for it: dA has freed this tile's V slot
            // without any arrival from this step, so the next phases of its barrier may be complete already.
            ok = __all_sync(0xffffffffu,
                            more ? wait_two(&ctl->bar_dp_full, G & 1, &ctl->bar_v_full[(G + 1) % VR],
                                            ((G + 1) / VR) & 1, ctx, ctl)
                                 : wait_or_abort(&ctl->bar_dp_full, G & 1, ctx, ctl));
            if (!ok) break;
            tc_fence_after();
            tmem_ld32(tl + kColDP + 32 * cq, dp);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 x = mul2(make_float2(p[2 * c], p[2 * c + 1]),
                                  sub2(make_float2(dp[2 * c], dp[2 * c + 1]), make_float2(delta[m], delta[m])));
            p[2 * c] = x.x, p[2 * c + 1] = x.y;
          }
          if (word != 0xffffffffu) {
            // keys outside the mask, or past the end: dS = 0 whatever their rows hold
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((word >> c) & 1u)) p[c] = 0.f;
          }
          store_packed32(tS + m * kTile, p);
          tc_fence_before();
          named_arrive(m == 0 ? kBarP : kBarDS, kBarCount);
        }
        if (!ok) {
          if (!met) named_sync(kBarP, kBarCount);
          named_sync(kBarDS, kBarCount);
        }
      }
      G0 += n;
      // epilogue: dQ = scale * (dS K)
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dq_done, it & 1, ctx, ctl));
      ++it;
      if (!ok) continue;
      tc_fence_after();
      const float cs = cq >= 2 && load_lambda(lam, lam_bf16, w.h) > 0.f ? -scale : scale;
      const uint32_t cQ = tl + kColDQ + cq * (D / 4) + (D == 64 ? (cq >> 1) * 64 : 0);
      const int i0 = w.t * kTile + (warp & 3) * 32;
      store_rows<D / 32>(dq, (((size_t)w.b * Sq + i0) * H + w.h) * D + cq * (D / 4), (size_t)H * D, Sq - i0, cQ, cs, false,
                         lane, ctx, q_extent);
      tc_fence_before();
      mbar_arrive(&ctl->bar_dq_free);
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
    for (int s = 0; s < KR; ++s)
      if (k_armed[s]) settle(&ctl->bar_k_full[s], (k_armed[s] - 1) & 1, ctx);
    for (int s = 0; s < VR; ++s)
      if (v_armed[s]) settle(&ctl->bar_v_full[s], (v_armed[s] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  await_previous();  // the dK/dV kernel
}

template <typename K>
int prepare(K kern, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess)
    return set_error(UAA_ERR_CUDA, "uaa_diff_attn_bwd: smem attribute: %s", cudaGetErrorString(e));
  return UAA_OK;
}

// Launches a kernel that may start as soon as all blocks of the one before it on the stream allow it.
template <typename K, typename... Args>
int launch_next(const char* what, K kern, int grid, int smem, cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

template <int D, bool kMask>
int launch_bwd(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const void* out,
               const void* out2, const void* dout, const float* lse, const uint8_t* mask, void* dq, void* dk, void* dv,
               void* dlam, int B, int Sq, int Sk, int H, float scale, float* rows, cudaStream_t s) {
  using bf = __nv_bfloat16;
  const int steps = steps_of(Sq);
  float* part = rows + row_floats(B, Sq, H);
  float* rest = part + (size_t)B * H * steps;
  const long long items_k = (long long)tiles_of(Sk) * H * B, items_q = (long long)tiles_of(Sq) * H * B;
  const long long row_blocks = (long long)B * steps * H;
  if (items_k > INT32_MAX || items_q > INT32_MAX || row_blocks > INT32_MAX)
    return set_error(UAA_ERR_UNSUPPORTED, "uaa_diff_attn_bwd: too many work items");
  DevCtx ctx;
  SegMaps mq, mk, mv, mdo;
  const SeqDesc qd = seq_plain(Sq), kd = seq_plain(Sk);
  int st;
  if ((st = get_dev_ctx(&ctx)) || (st = encode_seq_maps(&mq, q, qd, B, H, D, kTile)) ||
      (st = encode_seq_maps(&mk, k, kd, B, H, D, kTile)) || (st = encode_seq_maps(&mv, v, kd, B, H, D, kTile)) ||
      (st = encode_seq_maps(&mdo, dout, qd, B, H, D, kTile)))
    return st;
  diff_rows_kernel<D><<<(int)row_blocks, kRowThreads, 0, s>>>(static_cast<const bf*>(out), static_cast<const bf*>(out2),
                                                             static_cast<const bf*>(dout), lse, lam, lam_bf16, rows,
                                                             part, B, Sq, H, ctx);
  if ((st = check_launch("uaa_diff_attn_bwd (rows)"))) return st;
  const int sms = device_sms();
  // with a key mask the heads go innermost while one batch's Q and dO fit in half of L2, so that the empty key
  // tiles spread evenly over the CTAs (as in the plain backward)
  const int head_inner = mask != nullptr && 4LL * H * Sq * D <= (64LL << 20);
  auto dkdv = diff_dkdv_kernel<D, kMask>;
  if ((st = prepare(dkdv, DkdvLayout<D>::kSmem)) ||
      (st = launch_next("uaa_diff_attn_bwd (dK/dV)", dkdv, (int)(items_k < sms ? items_k : sms), DkdvLayout<D>::kSmem, s,
                        mq.m[0], mk.m[0], mv.m[0], mdo.m[0], lam, lam_bf16, rows, mask, static_cast<bf*>(dk),
                        static_cast<bf*>(dv), rest, B, H, Sq, Sk, (int)items_k, head_inner, scale, scale * kLog2e, ctx)))
    return st;
  // dQ's rounds: the CTAs on the `late` SMs that the last round of dK/dV keeps busy start one dK/dV item later, which is
  // worth 1.66 (D = 64: 1.33) dQ items of as many tiles, and take that much less.  Whole backward with equal shares and
  // this way: B = 2, Sq = 4096, Sk = 512, H = 24, D = 128: 240 and 192 us; B = 2, S = 1024, H = 24, D = 64: 90 and 85 us
  const int grid_q = (int)(items_q < sms ? items_q : sms), late = (int)(items_k < sms ? items_k : items_k % sms);
  DqWalk walk{INT32_MAX, grid_q};
  if (late > 0 && late < grid_q) {
    const int early = grid_q - late;
    const double delay = (D == 128 ? 1.66 : 1.33) * tiles_of(Sq) / tiles_of(Sk);
    double best = 1e30;
    for (long long r = items_q / grid_q + 1, k = 0; r >= 1 && k < 64; --r, ++k) {
      const long long left = items_q - r * grid_q;
      const double end = std::max(delay + r, (double)(r + (left > 0 ? (left + early - 1) / early : 0)));
      if (end < best) best = end, walk = DqWalk{(int)r, early};
    }
  }
  auto dqk = diff_dq_kernel<D, kMask>;
  if ((st = prepare(dqk, DqLayout<D>::kSmem))) return st;
  return launch_next("uaa_diff_attn_bwd (dQ)", dqk, grid_q, DqLayout<D>::kSmem, s, mq.m[0],
                     mk.m[0], mv.m[0], mdo.m[0], lam, lam_bf16, rows, mask, static_cast<bf*>(dq), part, rest, dlam, B, H, Sq,
                     Sk, (int)items_q, walk, scale, scale * kLog2e, ctx);
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" size_t uaa_diff_attn_bwd_workspace_bytes(int B, int Sq, int Sk, int H, int D) {
  if (B < 0 || Sq < 0 || Sk < 0 || H < 0 || (D != 64 && D != 128)) return 0;
  // the row vectors, the sums of 64 rows' Delta_2, and a sum per 128 keys
  return ((row_floats(B, Sq, H) + (size_t)B * H * (steps_of(Sq) + tiles_of(Sk))) * 4 + 255) & ~(size_t)255;
}

extern "C" int uaa_diff_attn_bwd(const void* q, const void* k, const void* v, const void* lambda, int lambda_dtype,
                                 const void* out, const void* out2, const void* dout, const float* lse,
                                 const uint8_t* key_mask, void* dq, void* dk, void* dv, void* dlambda, int B, int Sq,
                                 int Sk, int H, int D, float scale, void* workspace, size_t workspace_bytes,
                                 uaa_stream_t stream) {
  const char* fn = "uaa_diff_attn_bwd";
  int st = validate_attn_sizes(fn, B, Sq, Sk, H, D, scale);
  if (st) return st;
  if (H == 0) return UAA_OK;
  if (B == 0 || (uint64_t)Sq + Sk == 0) {  // no row: the sum over them is 0
    if ((st = check_lambda(fn, dlambda, lambda_dtype))) return st;
    const cudaError_t e = cudaMemsetAsync(dlambda, 0, (size_t)H * (lambda_dtype == UAA_BF16 ? 2 : 4),
                                          static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    return UAA_OK;
  }
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
  const size_t need = uaa_diff_attn_bwd_workspace_bytes(B, Sq, Sk, H, D);
  if (workspace_bytes < need)
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  auto go = D == 64 ? (key_mask ? launch_bwd<64, true> : launch_bwd<64, false>)
                    : (key_mask ? launch_bwd<128, true> : launch_bwd<128, false>);
  return go(q, k, v, lambda, lambda_dtype == UAA_BF16, out, out2, dout, lse, key_mask, dq, dk, dv, dlambda, B, Sq, Sk,
            H, scale, static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
}
