// Differential attention, forward (the formulas stand in diff_shared.cuh): two
// kernels, one for tiles of 128 query rows on the tensor cores, one for a few
// query rows against many keys, which is bound by reading K and V.
//
// Tiles.  A persistent CTA per SM walks items; an item is one 128-row query tile
// of one (batch, head), both maps, against tiles of 80 keys (D = 64: 128).
//   warp 8     TMA: the item's Q tile (two buffers), then K_j, V_j through a
//              ring; V_j is loaded once and read by both maps.
//   warp 9     tcgen05, one elected lane:
//                S1_0 S2_0 | S1_1 | S2_1 | PV1_0 | S1_2 | PV2_0 | S2_2 | PV1_1 | ...
//              S_m = Q_m K_m^T takes D/2 columns (half the steps of a full
//              product), PV_m reads P_m from TMEM and V from shared memory.
//   warps 0-3  softmax of map 1, warps 4-7 of map 2: a thread owns a query row
//              (a TMEM lane), one pass with a running maximum; the accumulator
//              is rescaled only when the maximum grew by more than 2^8.
//   warps 10, 11  wait for copies and products on behalf of map 1 and map 2.
//   epilogue   the warpgroups exchange 1/l_1 and 1/l_2 through shared memory and
//              round half of the columns each into shared memory, over the item's
//              Q, whose last product is done: O_2, which every warp reads back in
//              whole lines and stores, then O, which warp 10 sends out by TMA.
//              (Stored from the registers, a row's 16 bytes a lane, every store
//              touches 32 lines.)
// P_m has columns of its own, so S_m of the next tile is formed as soon as the
// warpgroup has read this one's, and a map's loop is its softmax alone.  That is
// what 80 keys are for at D = 128: with 128 the two S and the two O fill TMEM,
// P_m lies over S_m, and every tile waits for PV_m and the next S_m in turn.
// Time at B = 1, S = 8191, H = 24, D = 128 (and at B = 2, Sq = 4096, Sk = 777 with a
// key mask): 960 us (128) that way; 980 (124) with columns of its own for P_m; 795
// (104) with the relay warps; 779 (86) with the outputs sent out of shared memory,
// 0.7 of it tensor time at the issue rate of 51 to 64 cycles a product.  What bounds
// the loop now is the issuer, whose bursts of four or five
// products stand 160 to 300 cycles apart.
// TMEM: S_1, S_2, P_1, P_2 from column 0; O_1, O_2 in the last 2 D.
// Keys outside the mask get P = 0; their rows of V are zeroed in shared memory
// before the product reads them, so an infinity or a NaN there leaves no trace.
#include <cooperative_groups.h>
#include <float.h>

#include "diff_shared.cuh"

namespace uaa {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Tiles of 128 query rows
constexpr int kThreads = 384;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kRelayWarp = 10;  // + m
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Named barriers.  For the issuer, from a map's warpgroup and relay warp: kBarS + m: S_m has been read and the next K
// tile has landed; kBarP + m: P_m is in TMEM and the V tile has landed.  For a warpgroup, from its relay warp: kBarF + m:
// S_m is complete and the V tile has landed; kBarE + m: P's buffer is free.  kBarL: the two warpgroups exchange their
// sums.  kBarO: O lies in shared memory.
constexpr uint32_t kBarS = 1, kBarP = 3, kBarIssue = 128 + 32 + 32;
constexpr uint32_t kBarF = 5, kBarE = 7, kBarRelay = 128 + 32;
constexpr uint32_t kBarL = 9, kBarO = 10, kBarOut = 256 + 32;

template <int D>
struct FwdLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kKeys = D == 128 ? 80 : 128;  // keys of a tile
  static constexpr int kWords = (kKeys + 31) / 32;
  static constexpr int kKeyBytes = kKeys * D * 2;  // a K or V tile
  static constexpr int kKeyChunk = kKeys * 128;    // 64 columns of it
  static constexpr int kRing = 8;
  static constexpr int kQ = 0;  // two Q tiles, each of them its item's O_2 and O at the end
  static constexpr int kRingOff = kQ + 2 * kTileBytes;
  static constexpr int kCtl = kRingOff + kRing * kKeyBytes;
  __host__ __device__ static constexpr uint32_t col_s(int m) { return kKeys * m; }
  __host__ __device__ static constexpr uint32_t col_p(int m) { return 2 * kKeys + kKeys / 2 * m; }
  __host__ __device__ static constexpr uint32_t col_o(int m) { return 512 - 2 * D + D * m; }
  static_assert(3 * kKeys <= 512 - 2 * D, "S, P and O of both maps exceed TMEM");
  // the bits of a full tile in mask word t
  __host__ __device__ static constexpr uint32_t full(int t) {
    return kKeys - 32 * t >= 32 ? 0xffffffffu : (1u << (kKeys - 32 * t)) - 1u;
  }
  static constexpr int kSum = kCtl + 512;          // 1/l of both maps, per row
  static constexpr int kCnt = kSum + 2 * 128 * 4;  // attended key tiles per mask row
  static constexpr int kSmem = kCnt + kMaxCntRows * 4;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

struct FwdCtl {
  uint64_t bar_q_full[2], bar_q_empty[2];
  uint64_t bar_kv_full[8], bar_kv_empty[8];
  uint64_t bar_s_full[2], bar_pv_done[2];
  uint64_t bar_o_free, bar_final;
  uint32_t tmem_base;
  int abort;
  alignas(16) uint32_t mask_words[8][4];  // per ring slot (filled with the V tile)
};
static_assert(sizeof(FwdCtl) <= 512, "control block");

struct Item {
  int t, h, b;
};
__device__ __forceinline__ Item decode_item(int item, int tiles, int H) {
  Item it;
  it.t = item % tiles;
  const int bh = item / tiles;
  it.h = bh % H;
  it.b = bh / H;
  return it;
}

template <int D, bool kMask>
__global__ void __launch_bounds__(kThreads, 1)
    diff_fwd_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                          const void* __restrict__ lam, int lam_bf16, const uint8_t* __restrict__ key_mask, __nv_bfloat16* __restrict__ out,
                          __nv_bfloat16* __restrict__ out2, float* __restrict__ lse, int B, int H, int Sq, int Sk,
                          int num_items, float scale_log2, DevCtx ctx) {
  using L = FwdLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing, kKeys = L::kKeys, W = L::kWords;
  constexpr int kPieces = D / 16;  // 16-byte pieces of half a row
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, kKeys, false, false);
  constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, false, true);
  constexpr float kLn2 = 0.6931471805599453f;

  extern __shared__ __align__(1024) uint8_t smem[];
  FwdCtl* ctl = reinterpret_cast<FwdCtl*>(smem + L::kCtl);
  float* sSum = reinterpret_cast<float*>(smem + L::kSum);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    // the swizzled operand tiles need 1024-byte alignment; never expected to trigger
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nqt = tiles_of(Sq);
  const int nkt = (Sk + kKeys - 1) / kKeys;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->bar_q_full[s], 1);
      mbar_init(&ctl->bar_q_empty[s], 1);
      mbar_init(&ctl->bar_s_full[s], 1);
      mbar_init(&ctl->bar_pv_done[s], 1);
    }
    for (int s = 0; s < R; ++s) {
      mbar_init(&ctl->bar_kv_full[s], 1);
      mbar_init(&ctl->bar_kv_empty[s], 1);
    }
    mbar_init(&ctl->bar_o_free, 256);
    mbar_init(&ctl->bar_final, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  // Attended key tiles per mask row: every role takes its tile count from this table, which no
  // one writes after the start, so all walk the same schedule, after a failure too.
  int* tile_cnt = reinterpret_cast<int*>(smem + L::kCnt);
  const bool skip = kMask && B <= kMaxCntRows;
  if (skip) {
    for (int r = threadIdx.x; r < B; r += kThreads) tile_cnt[r] = 0;
    __syncthreads();
    const int pairs = B * nkt;
    for (int p0 = warp * 4; p0 < pairs; p0 += (kThreads / 32) * 4) {
      bool any[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pr = p0 + u;
        bool hit = false;
        if (pr < pairs) {
          const int r = pr / nkt, k0 = (pr - r * nkt) * kKeys;
          const uint8_t* row = key_mask + (size_t)r * Sk + k0;
#pragma unroll
          for (int t = 0; t < W; ++t) {
            const int c = 32 * t + lane;
            hit |= c < kKeys && k0 + c < Sk && row[c] != 0;
          }
        }
        any[u] = hit;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (__any_sync(0xffffffffu, any[u]) && lane == 0 && p0 + u < pairs) atomicAdd(&tile_cnt[(p0 + u) / nkt], 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t o_extent = (size_t)B * Sq * H * D, lse_extent = (size_t)B * H * 2 * Sq;
  auto item_tiles = [&](int b) { return skip ? tile_cnt[b] : nkt; };

  uint32_t kv_armed[8] = {}, q_armed[2] = {};  // uses armed per barrier, for the teardown
  bool mma_issued = false;                     // set in the issuing lane once it has issued an MMA

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t n = 0;   // K/V ring counter across items
    uint32_t ne = 0;  // items with at least one attended key tile
    for (int item = blockIdx.x; ok && item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H);
      if (item_tiles(w.b) == 0) continue;
      const int qs = ne & 1;
      if (lane == 0) {
        if (ne > 1) ok = wait_or_abort(&ctl->bar_q_empty[qs], ((ne >> 1) - 1) & 1, ctx, ctl);
        if (ok) {
          mbar_arrive_expect_tx(&ctl->bar_q_full[qs], L::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_load_4d(smem + L::kQ + qs * L::kTileBytes + c * kChunkBytes, &tmQ, &ctl->bar_q_full[qs], c * 64, w.h,
                        w.t * kTile, w.b);
          q_armed[qs] = (ne >> 1) + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++ne;
      // the mask bytes of a tile, a lane's of each word, read one tile ahead: their latency is longer than a tile's time
      uint8_t bytes[W];
      auto read_mask = [&](int j) {
#pragma unroll
        for (int t = 0; t < W; ++t) {
          const int c = j * kKeys + 32 * t + lane;
          bytes[t] = 32 * t + lane < kKeys && c < Sk ? key_mask[(size_t)w.b * Sk + c] : (uint8_t)0;
        }
      };
      if (kMask) read_mask(0);
      for (int j = 0; ok && j < nkt; ++j) {
        uint32_t words[4] = {0u, 0u, 0u, 0u};  // bit c of word t: key 32t + c of the tile is attended
        if (kMask) {
#pragma unroll
          for (int t = 0; t < W; ++t) words[t] = __ballot_sync(0xffffffffu, bytes[t] != 0);
          read_mask(j + 1);
          if (skip && (words[0] | words[1] | words[2] | words[3]) == 0) continue;
        }
#pragma unroll
        for (int kind = 0; kind < 2; ++kind, ++n) {  // 0 = K_j, 1 = V_j
          const int slot = n % R;
          const uint32_t use = n / R;
          if (lane == 0 && use > 0) ok = wait_or_abort(&ctl->bar_kv_empty[slot], (use - 1) & 1, ctx, ctl);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (kMask && kind == 1 && lane == 0) {
#pragma unroll
            for (int t = 0; t < W; ++t) ctl->mask_words[slot][t] = words[t];
          }
          if (lane == 0 && (int)n != ctx.drop_load) {
            mbar_arrive_expect_tx(&ctl->bar_kv_full[slot], L::kKeyBytes);
            const CUtensorMap* map = kind == 0 ? &tmK : &tmV;
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(smem + L::kRingOff + slot * L::kKeyBytes + c * L::kKeyChunk, map, &ctl->bar_kv_full[slot],
                          c * 64, w.h, j * kKeys, w.b);
            kv_armed[slot] = use + 1;
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the schedule and computes the descriptors, one elected lane waits and
    // issues.  Within an item this warp waits on named barriers only.
    uint32_t el_lane;
    const bool el = elect_one_sync(&el_lane);
    bool ok = true;
    uint32_t g = 0;   // key tiles across items (phase index of s / pv barriers)
    uint32_t ne = 0;  // items with at least one attended key tile
    auto ring_addr = [&](uint32_t n) { return sbase + L::kRingOff + (n % R) * L::kKeyBytes; };
    // byte offset of 16-column step kk of map m in a K tile (map_step in a Q tile, whose chunks are longer)
    auto key_step = [](int m, int kk) {
      const int col = m * (D / 2) + 16 * kk;
      return (uint32_t)((col / 64) * L::kKeyChunk + (col % 64) * 2);
    };
    // S_m of key tile t; the second map's releases K's slot
    auto issue_s = [&](int m, uint32_t t, uint32_t qs) {
      const uint64_t a0 = sdesc_sw128(sbase + L::kQ + qs * L::kTileBytes, 16, 1024);
      const uint64_t b0 = sdesc_sw128(ring_addr(2 * t), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const uint64_t a = desc_add(a0, m == 0 ? map_step<D>(0, kk) : map_step<D>(1, kk));
        const uint64_t b = desc_add(b0, key_step(m, kk));
        if (el) mma_ss_checked(mg, tmem + L::col_s(m), a, b, kIdescS, kk > 0, kKeys);
      }
      if (el) {
        mma_commit(&ctl->bar_s_full[m]);
        if (m == 1) mma_commit(&ctl->bar_kv_empty[(2 * t) % R]);
      }
    };
    // O_m += P_m V_t; the second map's releases V's slot
    auto issue_pv = [&](int m, uint32_t t, bool first) {
      const uint64_t b0 = sdesc_sw128(ring_addr(2 * t + 1), L::kKeyChunk, 1024);
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk) {
        const uint64_t b = desc_add(b0, kk * 2048);
        if (el)
          mma_ts_checked(mg, tmem + L::col_o(m), tmem + L::col_p(m) + kk * 8, b, kIdescPV, (!first || kk > 0) ? 1u : 0u,
                         D);
      }
      if (el) {
        mma_commit(&ctl->bar_pv_done[m]);
        if (m == 1) mma_commit(&ctl->bar_kv_empty[(2 * t + 1) % R]);
      }
    };
    for (int item = blockIdx.x; item < num_items; item += gridDim.x) {
      const int nt = item_tiles(decode_item(item, nqt, H).b);
      if (nt == 0) continue;
      // After a failure anywhere in the CTA this warp stops issuing but still meets the softmax
      // warpgroups at every named barrier of the schedule.
      if (ok && *reinterpret_cast<volatile int*>(&ctl->abort)) ok = false;
      const uint32_t qs = ne & 1;
      if (ok) {
        bool w = true;
        if (el) {
          w = wait_or_abort(&ctl->bar_q_full[qs], (ne >> 1) & 1, ctx, ctl);
          if (w) w = wait_or_abort(&ctl->bar_kv_full[(2 * g) % R], ((2 * g) / R) & 1, ctx, ctl);
        }
        ok = __shfl_sync(0xffffffffu, w, el_lane);
        if (ok) {
          tc_fence_after();
          issue_s(0, g, qs);
          issue_s(1, g, qs);
          if (el) mma_issued = true;
        }
      }
      for (int j = 0; j <= nt; ++j) {
        const uint32_t t = g + j;
        const bool more = j + 1 < nt;
        // A product's operands have landed when its barrier passes: the warpgroups waited for them.
        if (j < nt) {
          named_sync(kBarS + 0, kBarIssue);
          if (ok && more) {
            tc_fence_after();
            issue_s(0, t + 1, qs);
          }
          __syncwarp();
        }
        if (j > 0) {
          named_sync(kBarP + 1, kBarIssue);
          if (ok) {
            tc_fence_after();
            issue_pv(1, t - 1, j == 1);
          }
          __syncwarp();
        }
        if (j < nt) {
          named_sync(kBarS + 1, kBarIssue);
          if (ok && more) {
            tc_fence_after();
            issue_s(1, t + 1, qs);
          }
          __syncwarp();
          named_sync(kBarP + 0, kBarIssue);
          if (ok && j == 0 && ne > 0) {
            // the previous item's epilogue must have read O before PV1_0 overwrites it
            bool w = true;
            if (el) w = wait_or_abort(&ctl->bar_o_free, (ne - 1) & 1, ctx, ctl);
            ok = __shfl_sync(0xffffffffu, w, el_lane);
          }
          if (ok) {
            tc_fence_after();
            issue_pv(0, t, j == 0);
          }
          __syncwarp();
        }
      }
      g += nt;
      ++ne;
    }
  } else if (warp >= kRelayWarp) {
    // ------------------------------------------------------------ relay warps
    // All waits for copies and products of map m's loop: a test of an mbarrier takes 150 to 300 cycles beside the
    // matrix instructions' shared-memory reads, even when it passes, and a named barrier about 30; so this warp does
    // the first and the softmax warps only the second.  After a failure it keeps meeting the others, one
    // rendezvous after the other.
    // Map 1's also sends O out at the end of an item.  The copy has left the Q tile, which the producer may then fill,
    // before the next item has come to its first P.
    const int m = warp - kRelayWarp;
    bool ok = true;
    uint32_t g = 0, ne = 0;  // key tiles, and items with at least one
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar, phase & 1, ctx, ctl));
    };
    auto meet = [&](uint32_t id, uint32_t count) {
      if (ok)
        named_arrive(id, count);
      else
        named_sync(id, count);
    };
    for (int item = blockIdx.x; item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H);
      const int nt = item_tiles(w.b);
      if (nt == 0) continue;
      for (int j = 0; j < nt; ++j) {
        const uint32_t gj = g + j, nv = 2 * gj + 1, nk1 = nv + 1;
        // V_j first: it has mostly landed long before S_m is complete, and its mask words come with it
        wait(&ctl->bar_kv_full[nv % R], nv / R);
        wait(&ctl->bar_s_full[m], gj);
        meet(kBarF + m, kBarRelay);
        if (j + 1 < nt) wait(&ctl->bar_kv_full[nk1 % R], nk1 / R);
        meet(kBarS + m, kBarIssue);
        if (j > 0) {
          // PV_{j-1} has read P's buffer.  That also says that the last kBarP has been passed, so this warp's arrivals
          // on it cannot overtake.
          wait(&ctl->bar_pv_done[m], gj - 1);
          meet(kBarE + m, kBarRelay);
        }
        meet(kBarP + m, kBarIssue);
        if (m == 0 && j == 0 && ne > 0) {
          if (lane == 0) {
            bulk_wait_read_all();
            mbar_arrive(&ctl->bar_q_empty[(ne - 1) & 1]);
          }
          __syncwarp();
        }
      }
      if (m == 0) {
        named_sync(kBarO, kBarOut);
        if (lane == 0 && ok && !*reinterpret_cast<volatile int*>(&ctl->abort) &&
            guard_store(ctx, (((size_t)w.b * Sq + w.t * kTile) * H + w.h) * D, D, o_extent)) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            tma_store_4d(smem + L::kQ + (ne & 1) * L::kTileBytes + c * kChunkBytes, &tmO, c * 64, w.h, w.t * kTile,
                         w.b);
          bulk_commit_group();
        }
        __syncwarp();
      }
      g += nt;
      ++ne;
    }
    if (m == 0 && lane == 0) bulk_wait_read_all();  // shared memory is read until then
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int m = warp >> 2;                 // map
    const int row = (warp & 3) * 32 + lane;  // TMEM lane = query row within the tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tS = tl + L::col_s(m), tP = tl + L::col_p(m), tO = tl + L::col_o(m);
    bool ok = true;
    uint32_t g = 0, ne = 0;
    for (int item = blockIdx.x; item < num_items; item += gridDim.x) {
      const Item w = decode_item(item, nqt, H);
      const int nt = item_tiles(w.b);
      const int qi = w.t * kTile + row;
      const bool qvalid = qi < Sq;
      // this thread writes half of the row's columns: half m
      const size_t oo = (((size_t)w.b * Sq + (qvalid ? qi : 0)) * H + w.h) * D + m * (D / 2);
      const size_t lo = (((size_t)w.b * H + w.h) * 2 + m) * Sq + (qvalid ? qi : 0);
      const bool ostore = qvalid && guard_store(ctx, oo, D / 2, o_extent) && guard_store(ctx, lo, 1, lse_extent);
      if (nt == 0) {
        // no attended key for this batch: nothing to read, O = O2 = 0 and LSE = -inf
        if (ostore) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            *reinterpret_cast<uint4*>(out + oo + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
            if (out2) *reinterpret_cast<uint4*>(out2 + oo + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
          lse[lo] = -INFINITY;
        }
        continue;
      }
      float mu = -INFINITY;  // log2-domain offset in use (scaled max, possibly stale by < 2^8)
      float l_run = 0.f;
      for (int j = 0; j < nt; ++j) {
        const uint32_t gj = g + j, nv = 2 * gj + 1;
        named_sync(kBarF + m, kBarRelay);
        tc_fence_after();
        // the tile's mask words, asked for ahead of S: the answer takes as long
        uint4 words;
        if (kMask) words = *reinterpret_cast<const uint4*>(ctl->mask_words[nv % R]);
        float s[kKeys];
        tmem_ld32x2(tS, tS + 32, *reinterpret_cast<float(*)[64]>(&s[0]));
        if constexpr (kKeys == 128)
          tmem_ld32x2(tS + 64, tS + 96, *reinterpret_cast<float(*)[64]>(&s[64]));
        else
          tmem_ld16(tS + 64, *reinterpret_cast<float(*)[16]>(&s[64]));
        tc_fence_before();
        named_arrive(kBarS + m, kBarIssue);
        if (kMask) {
          const int vs = nv % R;
          const uint32_t mw[4] = {words.x, words.y, words.z, words.w};
          bool whole = true;
#pragma unroll
          for (int q = 0; q < W; ++q) whole = whole && mw[q] == L::full(q);
          if (!whole) {
#pragma unroll
            for (int c = 0; c < kKeys; ++c)
              if (!((mw[c >> 5] >> (c & 31)) & 1u)) s[c] = -INFINITY;
            // V_j's rows outside the mask: read as zeros by both maps' products, the second of which is
            // issued behind the first
            if (m == 0) {
              if (row < kKeys && !((ctl->mask_words[vs][row >> 5] >> lane) & 1u)) {
#pragma unroll
                for (int c = 0; c < kChunks * 8; ++c)
                  *reinterpret_cast<uint4*>(smem + L::kRingOff + vs * L::kKeyBytes + (c >> 3) * L::kKeyChunk +
                                            row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
          }
        } else if (j == nkt - 1 && Sk - j * kKeys < kKeys) {
#pragma unroll
          for (int c = 0; c < kKeys; ++c)
            if (c >= Sk - j * kKeys) s[c] = -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) m8[q] = fmaxf(s[q], s[q + 8]);
#pragma unroll
        for (int c = 16; c < kKeys; c += 16)
#pragma unroll
          for (int q = 0; q < 8; ++q) m8[q] = max3(m8[q], s[c + q], s[c + q + 8]);
        const float mt = fmaxf(max3(m8[0], m8[1], m8[2]), max3(max3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
        // -inf if every key of the tile is masked.  The offset stays finite: a score of +inf then gives P = l = +inf, so
        // LSE = +inf and, times 1/l = 0, a row of NaN; a NaN score, which a maximum passes over, gives P = l = NaN.
        const float mt2 = fminf(mt * scale_log2, FLT_MAX);
        float alpha = 1.f;
        if (mt2 > mu + kRescaleThreshold) {
          alpha = ex2(mu - mt2);  // 0 when mu = -inf
          mu = mt2;
        }
        const float mu_use = (mu == -INFINITY) ? 0.f : mu;
        const float2 c2 = make_float2(scale_log2, scale_log2);
        const float2 nm2 = make_float2(-mu_use, -mu_use);
        float2 rs2 = make_float2(0.f, 0.f);
        uint32_t pk[kKeys / 2];
#pragma unroll
        for (int c = 0; c < kKeys / 2; ++c) {
          const float2 x = fma2(make_float2(s[2 * c], s[2 * c + 1]), c2, nm2);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          rs2 = add2(rs2, e);
          pk[c] = pack_bf16(e.x, e.y);
        }
        l_run = l_run * alpha + (rs2.x + rs2.y);
        if (j > 0) named_sync(kBarE + m, kBarRelay);  // PV_{j-1} is done: P's buffer is free, and O may be rescaled
        tc_fence_after();
        tmem_st32_bits(tP, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
        if constexpr (kKeys == 128)
          tmem_st32_bits(tP + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
        else
          tmem_st8_bits(tP + 32, *reinterpret_cast<const uint32_t(*)[8]>(&pk[32]));
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(tO + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(tO + 32 * c, o);
          }
        }
        tc_fence_before();
        named_arrive(kBarP + m, kBarIssue);
      }
      if (ok) {
        bool okw = wait_or_abort(&ctl->bar_pv_done[0], (g + nt - 1) & 1, ctx, ctl);
        if (okw) okw = wait_or_abort(&ctl->bar_pv_done[1], (g + nt - 1) & 1, ctx, ctl);
        ok = __all_sync(0xffffffffu, okw);
      }
      // both maps' products are done, which the previous item's readers of these sums allowed (bar_o_free)
      sSum[m * kTile + row] = l_run == 0.f ? 0.f : 1.f / l_run;
      named_sync(kBarL, 256);
      const uint32_t qs = ne & 1;
      g += nt;
      ++ne;
      if (!ok) {
        named_arrive(kBarO, kBarOut);
        continue;
      }
      tc_fence_after();
      const float c1 = sSum[row], c2 = sSum[kTile + row];
      const float lm = load_lambda(lam, lam_bf16, w.h);
      // this warp's 32 rows and half of the columns, in 16-byte pieces of the swizzled tile
      auto at = [&](int r, int i) {
        const int piece = m * kPieces + i;
        return reinterpret_cast<uint4*>(smem + L::kQ + qs * L::kTileBytes + (piece >> 3) * kChunkBytes + r * 128 +
                                        (((piece ^ r) & 7) << 4));
      };
      auto put = [&](int i, const float* x, float c) {
        *at(row, i) = make_uint4(pack_bf16(x[0] * c, x[1] * c), pack_bf16(x[2] * c, x[3] * c),
                                 pack_bf16(x[4] * c, x[5] * c), pack_bf16(x[6] * c, x[7] * c));
      };
      if (out2) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float o[32];
          tmem_ld32(tl + L::col_o(1) + m * (D / 2) + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) put(4 * c + i, o + 8 * i, c2);
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < kPieces; ++x) {
          const int r = (warp & 3) * 32 + x * (32 / kPieces) + lane / kPieces, i = lane % kPieces;
          const uint4 v = *at(r, i);
          const size_t o = (((size_t)w.b * Sq + w.t * kTile + r) * H + w.h) * D + m * (D / 2) + 8 * i;
          if (w.t * kTile + r < Sq && guard_store(ctx, o, 8, o_extent)) *reinterpret_cast<uint4*>(out2 + o) = v;
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        float o[64];  // 32 columns of O1, then of O2
        tmem_ld32x2(tl + L::col_o(0) + m * (D / 2) + 32 * c, tl + L::col_o(1) + m * (D / 2) + 32 * c, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = o[i] * c1 - lm * (o[32 + i] * c2);
#pragma unroll
        for (int i = 0; i < 4; ++i) put(4 * c + i, o + 8 * i, 1.f);
      }
      fence_proxy_async_smem();
      named_arrive(kBarO, kBarOut);
      tc_fence_before();
      mbar_arrive(&ctl->bar_o_free);
      if (ostore) lse[lo] = l_run == 0.f ? -INFINITY : mu * kLn2 + logf(l_run);
    }
  }

  // ------------------------------------------------------------ teardown
  // Waits here ignore the abort flag (they must see in-flight work land) but stay bounded.
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp && mma_issued) {
    mma_commit(&ctl->bar_final);
    settle(&ctl->bar_final, 0, ctx);
  }
  if (warp == kProducerWarp && lane == 0) {
    for (int s = 0; s < 2; ++s)
      if (q_armed[s]) settle(&ctl->bar_q_full[s], (q_armed[s] - 1) & 1, ctx);
    for (int s = 0; s < R; ++s)
      if (kv_armed[s]) settle(&ctl->bar_kv_full[s], (kv_armed[s] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kMask>
int launch_tiles(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const uint8_t* mask,
                 void* out, void* out2, float* lse, int B, int Sq, int Sk, int H, float scale, cudaStream_t s) {
  const char* fn = "uaa_diff_attn_fwd";
  DevCtx ctx;
  SegMaps mq, mk, mv, mo;
  int st;
  if ((st = get_dev_ctx(&ctx)) || (st = encode_seq_maps(&mq, q, seq_plain(Sq), B, H, D, kTile)) ||
      (st = encode_seq_maps(&mk, k, seq_plain(Sk), B, H, D, FwdLayout<D>::kKeys)) ||
      (st = encode_seq_maps(&mv, v, seq_plain(Sk), B, H, D, FwdLayout<D>::kKeys)) ||
      (st = encode_seq_maps(&mo, out, seq_plain(Sq), B, H, D, kTile)))
    return st;
  auto kern = diff_fwd_tiles_kernel<D, kMask>;
  const int smem = FwdLayout<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: smem attribute: %s", fn, cudaGetErrorString(e));
  const long long items = (long long)tiles_of(Sq) * H * B;
  if (items > INT32_MAX) return set_error(UAA_ERR_UNSUPPORTED, "%s: too many work items", fn);
  const int grid = (int)(items < device_sms() ? items : device_sms());
  kern<<<grid, kThreads, smem, s>>>(mq.m[0], mk.m[0], mv.m[0], mo.m[0], lam, lam_bf16, mask,
                                    static_cast<__nv_bfloat16*>(out), static_cast<__nv_bfloat16*>(out2), lse, B, H, Sq,
                                    Sk, (int)items, scale * kLog2e, ctx);
  return check_launch(fn);
}

// ---------------------------------------------------------------------------
// A few query rows against many keys
//
// Bound: reading K and V once (4 D bytes a key and head).  A cluster of CTAs
// shares one (batch, head) and NQ query rows: each CTA takes a run of keys, its
// warps take keys in turn, a row of K or V spread over D/8 lanes of 16 bytes, so
// a warp's load brings 256/D keys.  Every lane group keeps the running maximum
// and sum of the keys it saw (its own map's; the other map's probability comes
// from a shuffle) and the two products of its 8 columns; they are joined over
// the warp, the CTA and, through distributed shared memory, the cluster, in a
// fixed order: one launch, no workspace.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxCluster = 8;
// Keys in flight per lane: as many as leave two CTAs on an SM (B = 4, Sk = 16389, H = 24, D = 128: one row 158 us with 4,
// 134 with 8, 222 with 12; two rows 172 us with 4, 136 with 6, 390 with 8; these two now 118 and 127: 6.8 and
// 6.3 TB/s).
__host__ __device__ constexpr int row_unroll(int nq) { return nq == 1 ? 8 : 6; }

template <int D, int NQ>
struct RowPart {  // a CTA's (or warp's) share of NQ rows
  float mx[NQ][2], sum[NQ][2];
  float acc[NQ][2][D];
};

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <int D, int NQ, bool kMask>
__global__ void __launch_bounds__(kRowThreads) diff_fwd_rows_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    const void* __restrict__ lam, int lam_bf16, const uint8_t* __restrict__ mask, __nv_bfloat16* __restrict__ out,
    __nv_bfloat16* __restrict__ out2, float* __restrict__ lse, int B, int Sq, int Sk, int H, int cluster,
    float scale_log2, DevCtx ctx) {
  constexpr int G = D / 8;       // lanes of a row
  constexpr int KW = 32 / G;     // keys of a warp's load
  constexpr int kRowUnroll = row_unroll(NQ);
  constexpr float kLn2 = 0.6931471805599453f;
  using Part = RowPart<D, NQ>;
  extern __shared__ __align__(16) uint8_t raw[];
  Part* part = reinterpret_cast<Part*>(raw);  // one per warp; part[0] ends up holding the CTA's
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % G, m = sub >= G / 2;  // columns 8 sub .. 8 sub + 7, which belong to map m
  const int rank = blockIdx.x % cluster;
  const int groups = (Sq + NQ - 1) / NQ;
  const long long unit = blockIdx.x / cluster;
  const int i0 = (int)(unit % groups) * NQ;
  const int h = (int)(unit / groups % H), b = (int)(unit / groups / H);
  const int per = (Sk + cluster - 1) / cluster;
  const int j_end = min(Sk, (rank + 1) * per);
  constexpr int kStep = kRowWarps * KW;  // keys of one load by all warps

  float2 qv[NQ][4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    if (i0 + n < Sq) a = *reinterpret_cast<const uint4*>(q + (((size_t)b * Sq + i0 + n) * H + h) * D + 8 * sub);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qv[n][e] = bf2(w[e]);
      qv[n][e].x *= scale_log2;
      qv[n][e].y *= scale_log2;
    }
  }
  float mx[NQ], sum[NQ];
  float2 acc[NQ][2][4];  // [own map, other map]
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    mx[n] = -INFINITY;
    sum[n] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][x][e] = make_float2(0.f, 0.f);
  }
  const size_t kbase = ((size_t)b * Sk * H + h) * D + 8 * sub, kstride = (size_t)H * D;
  const uint8_t* mrow = kMask ? mask + (size_t)b * Sk : nullptr;
#pragma unroll 1
  for (int j0 = rank * per + warp * KW + lane / G; j0 - lane / G < j_end; j0 += kStep * kRowUnroll) {
    bool on[kRowUnroll];
    uint4 kr[kRowUnroll], vr[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const int j = j0 + u * kStep;
      on[u] = j < j_end && (!kMask || mrow[j] != 0);
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      // a key outside the mask is not read: whatever its rows hold leaves no trace
      kr[u] = vr[u] = make_uint4(0u, 0u, 0u, 0u);
      if (on[u]) {
        const size_t at = kbase + (size_t)(j0 + u * kStep) * kstride;
        kr[u] = __ldcs(reinterpret_cast<const uint4*>(k + at));
        vr[u] = __ldcs(reinterpret_cast<const uint4*>(v + at));
      }
    }
    float s[NQ][kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const uint32_t w[4] = {kr[u].x, kr[u].y, kr[u].z, kr[u].w};
      float2 kf[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) kf[e] = bf2(w[e]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float2 d = mul2(qv[n][0], kf[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) d = fma2(qv[n][e], kf[e], d);
        float x = d.x + d.y;
#pragma unroll
        for (int o = G / 4; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        s[n][u] = on[u] ? x : -INFINITY;
      }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = s[n][0];
#pragma unroll
      for (int u = 1; u < kRowUnroll; ++u) top = fmaxf(top, s[n][u]);
      if (__any_sync(0xffffffffu, top > mx[n])) {
        const float now = fminf(fmaxf(mx[n], top), FLT_MAX);  // finite, as in the tiles
        const float alpha = mx[n] == now ? 1.f : ex2(mx[n] - now);  // 0 from -inf
        mx[n] = now;
        sum[n] *= alpha;
        const float other = __shfl_xor_sync(0xffffffffu, alpha, G / 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[n][0][e] = mul2(acc[n][0][e], make_float2(alpha, alpha));
          acc[n][1][e] = mul2(acc[n][1][e], make_float2(other, other));
        }
      }
    }
    float base[NQ];  // 0 while every score was -inf, so that ex2(-inf - base) is 0
#pragma unroll
    for (int n = 0; n < NQ; ++n) base[n] = mx[n] == -INFINITY ? 0.f : mx[n];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const uint32_t w[4] = {vr[u].x, vr[u].y, vr[u].z, vr[u].w};
      float2 vf[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) vf[e] = bf2(w[e]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float p = ex2(s[n][u] - base[n]);  // a key outside the mask has a score of -inf
        const float o = __shfl_xor_sync(0xffffffffu, p, G / 2);
        sum[n] += p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[n][0][e] = fma2(make_float2(p, p), vf[e], acc[n][0][e]);
          acc[n][1][e] = fma2(make_float2(o, o), vf[e], acc[n][1][e]);
        }
      }
    }
  }
  // the warp's lane groups, then its share into shared memory
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float top = mx[n];
#pragma unroll
    for (int o = G; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float c = mx[n] == -INFINITY ? 0.f : ex2(mx[n] - top);
    const float oc = __shfl_xor_sync(0xffffffffu, c, G / 2);
    float l = sum[n] * c;
#pragma unroll
    for (int o = G; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (sub % (G / 2) == 0 && lane < G) {
      part[warp].mx[n][m] = top;
      part[warp].sum[n][m] = l;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 a = acc[n][x][e];
        const float f = x == 0 ? c : oc;
        a.x *= f;
        a.y *= f;
#pragma unroll
        for (int o = G; o < 32; o *= 2) {
          a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
          a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
        }
        if (lane < G) *reinterpret_cast<float2*>(&part[warp].acc[n][x == 0 ? m : 1 - m][8 * sub + 2 * e]) = a;
      }
  }
  __syncthreads();
  // the CTA's: every (row, map, column) by one thread, into registers, then over the first warp's share
  constexpr int kVals = NQ * 2 * D;
  constexpr int kPer = (kVals + kRowThreads - 1) / kRowThreads;
  float val[kPer];
  float cta_mx = -INFINITY, cta_sum = 0.f;
  auto factor = [](float w, float top) { return w == -INFINITY ? 0.f : ex2(w - top); };
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int at = threadIdx.x + x * kRowThreads;
    if (at < kVals) {
      const int n = at / (2 * D), mm = at / D % 2, c = at % D;
      float top = -INFINITY, a = 0.f;
      for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, part[w].mx[n][mm]);
      for (int w = 0; w < kRowWarps; ++w) a += part[w].acc[n][mm][c] * factor(part[w].mx[n][mm], top);
      val[x] = a;
    }
  }
  if (threadIdx.x < 2 * NQ) {
    const int n = threadIdx.x / 2, mm = threadIdx.x % 2;
    for (int w = 0; w < kRowWarps; ++w) cta_mx = fmaxf(cta_mx, part[w].mx[n][mm]);
    for (int w = 0; w < kRowWarps; ++w) cta_sum += part[w].sum[n][mm] * factor(part[w].mx[n][mm], cta_mx);
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    const int at = threadIdx.x + x * kRowThreads;
    if (at < kVals) part[0].acc[at / (2 * D)][at / D % 2][at % D] = val[x];
  }
  if (threadIdx.x < 2 * NQ) {
    part[0].mx[threadIdx.x / 2][threadIdx.x % 2] = cta_mx;
    part[0].sum[threadIdx.x / 2][threadIdx.x % 2] = cta_sum;
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  // the cluster's: rank r writes every cluster-th pair of columns
  const float lm = load_lambda(lam, lam_bf16, h);
  for (int at = rank * kRowThreads + threadIdx.x; at < NQ * (D / 2); at += cluster * kRowThreads) {
    const int n = at / (D / 2), c = at % (D / 2) * 2;
    if (i0 + n >= Sq) continue;
    float2 o[2];
    float lsum[2], top[2];
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      top[mm] = -INFINITY;
      lsum[mm] = 0.f;
      o[mm] = make_float2(0.f, 0.f);
      for (int r = 0; r < cluster; ++r) top[mm] = fmaxf(top[mm], cl.map_shared_rank(part, r)->mx[n][mm]);
      for (int r = 0; r < cluster; ++r) {
        const Part* p = cl.map_shared_rank(part, r);
        const float f = factor(p->mx[n][mm], top[mm]);
        const float2 a = *reinterpret_cast<const float2*>(&p->acc[n][mm][c]);
        lsum[mm] += p->sum[n][mm] * f;
        o[mm].x += a.x * f;
        o[mm].y += a.y * f;
      }
      const float inv = lsum[mm] == 0.f ? 0.f : 1.f / lsum[mm];
      o[mm].x *= inv;
      o[mm].y *= inv;
    }
    const size_t oo = (((size_t)b * Sq + i0 + n) * H + h) * D + c, o_extent = (size_t)B * Sq * H * D;
    if (!guard_store(ctx, oo, 2, o_extent)) continue;
    *reinterpret_cast<uint32_t*>(out + oo) = pack_bf16(o[0].x - lm * o[1].x, o[0].y - lm * o[1].y);
    if (out2) *reinterpret_cast<uint32_t*>(out2 + oo) = pack_bf16(o[1].x, o[1].y);
    if (c < 4) {  // columns 0 and 2 stand for the two maps
      const int mm = c / 2;
      const size_t lo = (((size_t)b * H + h) * 2 + mm) * Sq + i0 + n;
      if (guard_store(ctx, lo, 1, (size_t)B * H * 2 * Sq))
        lse[lo] = lsum[mm] == 0.f ? -INFINITY : top[mm] * kLn2 + logf(lsum[mm]);
    }
  }
  cl.sync();  // no CTA leaves while another reads its shared memory
}

template <int D, int NQ, bool kMask>
int launch_rows(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const uint8_t* mask,
                void* out, void* out2, float* lse, int B, int Sq, int Sk, int H, float scale, cudaStream_t s) {
  const char* fn = "uaa_diff_attn_fwd";
  DevCtx ctx;
  if (int st = get_check_ctx(&ctx)) return st;
  auto kern = diff_fwd_rows_kernel<D, NQ, kMask>;
  const int smem = kRowWarps * (int)sizeof(RowPart<D, NQ>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: smem attribute: %s", fn, cudaGetErrorString(e));
  const long long units = (long long)B * H * ((Sq + NQ - 1) / NQ);
  // as many CTAs per unit as fill the SMs twice (two are resident), each with at least two loads of keys per warp
  const int least = 2 * kRowWarps * (256 / D) * row_unroll(NQ);
  long long c = (4LL * device_sms() / units + 1) / 2;
  const long long most = (Sk + least - 1) / least;
  c = c > most ? most : c;
  const int cluster = c < 1 ? 1 : (c > kMaxCluster ? kMaxCluster : (int)c);
  if (units * cluster > INT32_MAX) return set_error(UAA_ERR_UNSUPPORTED, "%s: too many work items", fn);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * cluster));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                         static_cast<const __nv_bfloat16*>(v), lam, lam_bf16, mask, static_cast<__nv_bfloat16*>(out),
                         static_cast<__nv_bfloat16*>(out2), lse, B, Sq, Sk, H, cluster, scale * kLog2e, ctx);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return check_launch(fn);
}

template <int D, bool kMask>
int launch_fwd(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const uint8_t* mask,
               void* out, void* out2, float* lse, int B, int Sq, int Sk, int H, float scale, cudaStream_t s) {
  // Few rows or tiles?  Per 128 keys and head, reading them for two rows takes about 11 ns of the whole card (D = 128;
  // half of it with D = 64), and a wave of query tiles about 1.1 us: the first is the faster for up to 96 such pairs of
  // rows a wave.  Measured both ways at Sk = 16389, D = 128, us (rows, tiles): B H = 96, Sq = 2: 136, 158; Sq = 3: 279,
  // 158; B H = 24, Sq = 8: 117, 141; Sq = 16: 258, 141; B H = 8, Sq = 16: 115, 138; Sq = 32: 165, 138; D = 64,
  // B H = 24, Sq = 16: 138, 145; Sq = 32: 252, 145; B H = 1536, Sk = 1000, Sq = 2: 158, 144.  One row needs less of
  // the kernel: Sq = 1 there: 143, 146.
  const long long bh = (long long)B * H, groups = (Sq + 1) / 2, sms = device_sms();
  const long long waves = (bh * tiles_of(Sq) + sms - 1) / sms;
  const bool rows = Sq == 1 || groups * bh * D <= 12288 * waves;
  auto go = !rows ? launch_tiles<D, kMask> : Sq == 1 ? launch_rows<D, 1, kMask> : launch_rows<D, 2, kMask>;
  return go(q, k, v, lam, lam_bf16, mask, out, out2, lse, B, Sq, Sk, H, scale, s);
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" int uaa_diff_attn_fwd(const void* q, const void* k, const void* v, const void* lambda, int lambda_dtype,
                                 const uint8_t* key_mask, void* out, void* out2, float* lse, int B, int Sq, int Sk,
                                 int H, int D, float scale, uaa_stream_t stream) {
  const char* fn = "uaa_diff_attn_fwd";
  int st = validate_attn_sizes(fn, B, Sq, Sk, H, D, scale);
  if (st) return st;
  if ((uint64_t)B * Sq * H == 0) return UAA_OK;
  if ((st = check_dev_ptr(fn, "q", q)) || (st = check_dev_ptr(fn, "k", k)) || (st = check_dev_ptr(fn, "v", v)) ||
      (st = check_dev_ptr(fn, "out", out)) || (out2 && (st = check_dev_ptr(fn, "out2", out2))) ||
      (st = check_lambda(fn, lambda, lambda_dtype)) || (st = check_lse(fn, lse)))
    return st;
  auto go = D == 64 ? (key_mask ? launch_fwd<64, true> : launch_fwd<64, false>)
                    : (key_mask ? launch_fwd<128, true> : launch_fwd<128, false>);
  return go(q, k, v, lambda, lambda_dtype == UAA_BF16, key_mask, out, out2, lse, B, Sq, Sk, H, scale,
            static_cast<cudaStream_t>(stream));
}
