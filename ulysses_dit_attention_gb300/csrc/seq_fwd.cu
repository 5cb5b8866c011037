// Attention over packed sequences and over the pages of a cache, forward (the
// formulas stand in seq_shared.cuh).
//
// Rows.  The g query heads that share a key head are rows of one tile: row r of a
// tile of a sequence is head r % g of token r / g, so a tile of 128 rows holds
// TT = 128 / g tokens and K and V are read once for all of them.  An item is two
// tiles (a pair) of one sequence and key head, against tiles of 128 keys.
//
// Work.  A persistent CTA per SM; the items of all sequences in a row, weighed by
// the keys that they read plus what an item costs beside them, are cut into equal
// shares, one a CTA, in the middle of an item where it falls so: long prompts, many
// short ones and one token over a long past fill the card alike, and the lengths stay
// on the device (every CTA adds up the weights itself when it starts, about 3 us).
// The parts of an item that was cut go to the workspace, unnormalised, and a second
// kernel joins them in order.
//   warp 8     TMA producer: the item's Q tiles, then K_j, V_j through a ring
//   warp 9     tcgen05 issuer (one elected lane)
//   warps 0-3  softmax of slot 0, warps 4-7 of slot 1: thread r owns row r (a TMEM
//              lane); running maximum and sum, O rescaled only when the maximum grew
//              by more than 2^8; P goes over S as the next product's operand
//   warps 10, 11  wait, look at V and send the rows out on behalf of slots 0 and 1
// An item's two tiles take the two slots and read the same keys.  Where the second
// tile is empty (few new tokens) both slots work on the first one, slot 0 on the even
// key tiles and slot 1 on the odd ones, and are joined in the epilogue: without that
// the chain S, softmax, P V of one tile takes longer than its keys take to arrive.
//
// TMEM: S / P of the slots in columns 0 and 128, O in 256 and 256 + D.
//
// Keys outside a row's border get P = 0.  P V multiplies that 0 by what V holds, so in
// the tiles that the border crosses the relay warps look at V first: an infinity or a
// NaN there becomes a zero, and the epilogue adds it to the rows that do read it.
//
// Bound and times (GB300, bf16, on the device).  Long sequences: the matrix pipe; a
// step of a pair at D = 128 takes 1.44 us, four products of 128 x 128 x 128 and
// 32768 exponentials, 1.1 us of it products: 8192 x 8192, 24 heads, 516 us = 1600
// TFLOP/s; 16389 tokens, 40 / 8 heads, causal 1690 us = 1630; 2048 new tokens over
// 27280 keys in pages 718 us = 1540.  At D = 64 the exponentials weigh as much as the
// products: 8192 x 8192, 24 heads, 457 us = 900 TFLOP/s.  Short sequences: filling and
// draining, 4.4 us an item beside its steps (images of 300 to 1100 tokens, D = 64, 24
// heads: 82 us at 16 % of the matrix pipe).  New tokens: memory, 16 tokens over
// 222000 keys, 8 key heads: 164 us, 5.5 TB/s.
#include <float.h>

#include <atomic>

#include "seq_shared.cuh"

namespace uaa {
namespace {

constexpr int kChunkBytes = 128 * 128;  // 128 rows x 128 bytes: 64 columns of a tile, 128-byte swizzled
constexpr int kThreads = 384;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kRelayWarp = 10;  // + slot
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Named barriers.  kBarP + t, "P of slot t is in TMEM, and the next K has landed": its softmax warps and its relay warp
// arrive, the issuer syncs.  Between the softmax warps and the relay warp of a slot: kBarF + t, "S is complete and V has
// landed", behind the last step "O is complete"; kBarI + t, the next item; kBarOut + t, the rows lie in shared memory.
// kBarL, the slots' sums.
constexpr uint32_t kBarP = 1, kBarPCount = 128 + 32 + 32;
constexpr uint32_t kBarF = 3, kBarI = 5, kBarOut = 7, kBarRelay = 128 + 32;
constexpr uint32_t kBarL = 9;
template <int D>
struct FwdLayout {
  static constexpr int kRing = D == 128 ? 5 : 10;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kQ = 0;  // two Q tiles
  static constexpr int kRingOff = kQ + 2 * kTileBytes;
  static constexpr int kCtl = kRingOff + kRing * kTileBytes;
  static constexpr int kStat = kCtl + 512;  // maximum and sum of slot 1's rows
  static constexpr int kKept = kStat + 2 * 128 * 4;  // the share's sequences
  static constexpr int kJobs = kKept + kKeptSeqs * 16;  // two a slot
  static constexpr int kSmem = kJobs + 4 * 64;
  static_assert(kSmem <= 232448, "shared memory exceeds the per-CTA limit");
};

struct FwdCtl {
  uint64_t bar_q_full, bar_q_empty;
  uint64_t bar_kv_full[10], bar_kv_empty[10];
  uint64_t bar_s_full[2], bar_pv_done[2];
  uint64_t bar_o_free, bar_final;
  uint32_t tmem_base;
  int abort;
  uint32_t dirty[2];  // the last even and odd item with an infinity or a NaN taken out of V (a relay warp can be at V of
                      // the next item while the other slot is in this one's epilogue, but not at that of one further)
  alignas(16) uint32_t words[10][4];       // paged, per ring slot: keys whose page is there (filled with V)
};
static_assert(sizeof(FwdCtl) <= 512, "control block");

// The softmax warps take registers that the other four do not need: 256 x 200 + 128 x 96 of the 384 x 168 that the block is
// launched with, which the host makes sure of (the softmax warps would wait for ever otherwise).  It keeps spills out of
// their loop: 2048 tokens over 27280 keys 755 -> 729 us, 24 sequences in chunks 152 -> 145, 8192 tokens at D = 64 433 -> 425.
constexpr int kLaunchRegs = 168;
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 96;"); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }
static_assert(256 * 200 + 128 * 96 <= 384 * kLaunchRegs, "registers of the block");

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kHalf) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <bool kHalf>
__device__ __forceinline__ uint4 pack8(const float* x, float f) {
  return make_uint4(pack2<kHalf>(x[0] * f, x[1] * f), pack2<kHalf>(x[2] * f, x[3] * f), pack2<kHalf>(x[4] * f, x[5] * f),
                    pack2<kHalf>(x[6] * f, x[7] * f));
}
// 16-bit floats, two a word: whether one of them is an infinity or a NaN; and the word without them
template <bool kHalf>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  constexpr uint32_t e = kHalf ? 0x7c00u : 0x7f80u;
  return (w & e) == e || (w >> 16 & e) == e;
}
template <bool kHalf>
__device__ __forceinline__ uint32_t times0_plus(uint32_t w, uint32_t c) {
  if constexpr (kHalf) asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(c) : "r"(w), "r"(0u));
  else asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(c) : "r"(w), "r"(0u));
  return c;
}
template <bool kHalf>
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  constexpr uint32_t e = kHalf ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0u : w & 0xffffu) | ((w >> 16 & e) == e ? 0u : w & 0xffff0000u);
}

// ---------------------------------------------------------------------------
// Items: pairs of tiles
using Pairs = QueryRow<2>;
struct Item {
  bool split;    // the second tile is empty: the slots take the key tiles in turn
  int c, n[2];   // key tiles of the part, and of the slots
  int lo, hi;    // keys that the first row reads, and the last one
};
__device__ __forceinline__ Item item_of(const SeqArgs& a, const Walk<Pairs>& w) {
  Item it;
  const int TT = a.TT, t0 = 2 * w.at.p * TT;
  it.hi = keys_of(a.s, w.q, min(w.q.n, t0 + 2 * TT) - 1);
  it.lo = keys_of(a.s, w.q, t0);
  it.split = w.q.n <= t0 + TT;
  it.c = max(w.j1 - w.j0, 0);
  if (it.split) {
    it.n[0] = (it.c + 1) / 2;
    it.n[1] = it.c / 2;
  } else {
    // (a first tile that reads no key takes one all the same, masked: slot 1 may still be in the item before, and slot 0
    // without a step could not tell the phases of its barriers apart)
    it.n[0] = held_in(tiles_in(keys_of(a.s, w.q, t0 + TT - 1), kBN) - w.j0, min(1, it.c), it.c);
    it.n[1] = it.c;
  }
  return it;
}
// The key tile whose K slot slot 0 takes its rows out through: every S that reads it comes before slot 0's last P V (before
// slot 1's, where both work on the same tile and slot 0 waits for slot 1).
__device__ __forceinline__ int stage_k(const Item& it) { return (it.split ? it.c : it.n[0]) - 1; }

// What the softmax warps of a slot have to know of an item.
enum { kSplit = 1, kPart = 2, kJoin = 4, kFull = 8 };  // kFull: every token of the slot's tile is there
struct alignas(16) Job {
  int c, n;  // key tiles of the part (-1: no more items) and of the slot
  int j0, lo, hi, flags;
  uint32_t base;   // ring counter of the first K
  uint32_t stage;  // ring slot for the way out
  Seq q;
  int tok0, h;  // first token of the tile within the sequence, key head
  uint32_t ne;
};
static_assert(sizeof(Job) == 64, "jobs");

// ---------------------------------------------------------------------------
// The workspace: the CTAs' first places, then 2 parts a CTA: O (D, rows) and (maximum, sum) of every row.
struct Parts {
  Cut* first;
  Seq* seqs;  // of the shares, where they are too many for shared memory: CTA c's from its first sequence + c on
  float* o;
  float2* stat;
  int rows;  // of a part: 128 or 256
};
__host__ __device__ __forceinline__ int part_rows(long long rows) { return rows <= 128 ? 128 : 256; }

template <int D>
__device__ __forceinline__ float* part_o(const Parts& w, int slot) { return w.o + (size_t)slot * D * w.rows; }
__device__ __forceinline__ float2* part_stat(const Parts& w, int slot) { return w.stat + (size_t)slot * w.rows; }

// Row j of V of key head h, or NULL where its page is not there.
template <bool kPaged>
__device__ __forceinline__ const uint16_t* value_row(const SeqArgs& a, const Seq& q, int h, int j) {
  const uaa_seqs& s = a.s;
  const uint16_t* v = static_cast<const uint16_t*>(s.v) + (size_t)h * s.v_head;
  if constexpr (kPaged) {
    const int page = s.table[(size_t)q.k0 * s.width + j / s.page];
    if (page < 0 || page >= s.pages) return nullptr;
    return v + (size_t)page * s.v_page + (size_t)(j % s.page) * s.v_row;
  } else {
    return v + (size_t)(q.k0 + j) * s.v_row;
  }
}

template <int D, bool kPaged, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
    seq_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                   const __grid_constant__ SeqArgs a, const Parts parts,
                   float scale_log2, DevCtx ctx) {
  using L = FwdLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing;
  constexpr uint32_t kIdescS = idesc_f16_f32(128, kBN, false, false, kHalf);
  constexpr uint32_t kIdescPV = idesc_f16_f32(128, D, false, true, kHalf);
  constexpr float kLn2 = 0.6931471805599453f;

  extern __shared__ __align__(1024) uint8_t smem[];
  FwdCtl* ctl = reinterpret_cast<FwdCtl*>(smem + L::kCtl);
  float* sStat = reinterpret_cast<float*>(smem + L::kStat);
  Job* jobs = reinterpret_cast<Job*>(smem + L::kJobs);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    // the swizzled operand tiles need 1024-byte alignment; never expected to trigger
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const uaa_seqs& s = a.s;
  asm volatile("griddepcontrol.launch_dependents;");

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_q_full, 1);
    mbar_init(&ctl->bar_q_empty, 1);
    for (int i = 0; i < R; ++i) {
      mbar_init(&ctl->bar_kv_full[i], 1);
      mbar_init(&ctl->bar_kv_empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&ctl->bar_s_full[w], 1);
      mbar_init(&ctl->bar_pv_done[w], 1);
    }
    mbar_init(&ctl->bar_o_free, 256);
    mbar_init(&ctl->bar_final, 1);
    ctl->abort = 0;
    ctl->dirty[0] = ctl->dirty[1] = 0;
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
  const Share share = find_share<Pairs, kPaged, kThreads>(a, smem + L::kStat, smem + L::kKept, parts.seqs,
                                                          ctx.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) parts.first[cta] = share.from;
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t o_extent = (size_t)s.T * s.Hq * D, lse_extent = (size_t)s.Hq * s.T;

  uint32_t kv_armed[R] = {}, q_armed = 0;  // uses armed per barrier, for the teardown
  bool mma_issued = false;                 // set in the issuing lane once it has issued an MMA

  if (warp >= kProducerWarp) {
    give_registers();
    if (warp == kProducerWarp) {
      // ------------------------------------------------------------ producer
      bool ok = true;
      uint32_t n = 0;   // K/V ring counter across items
      uint32_t ne = 0;  // items with at least one key tile
      const int my_part = lane & 7, my_chunk = lane >> 3;  // paged: this lane's copy of a tile
      Walk<Pairs> w(share);
      while (ok && w.next(a)) {
        const Item it = item_of(a, w);
        if (it.c == 0) continue;
        const int h = w.at.h;
        if (lane == 0) {
          if (ne > 0) ok = wait_or_abort(&ctl->bar_q_empty, (ne - 1) & 1, ctx, ctl);
          if (ok) {
            const int tiles = it.split ? 1 : 2;
            mbar_arrive_expect_tx(&ctl->bar_q_full, tiles * kChunks * a.TT * a.g * 128);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(smem + L::kQ + t * L::kTileBytes + c * kChunkBytes, &tmQ, &ctl->bar_q_full, c * 64, 0, h,
                            w.q.q0 + (2 * w.at.p + t) * a.TT);
            q_armed = ne + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++ne;
        // Paged: the table's entries, a lane's of a window of 32 and of the next one, read long before they are needed
        const int per = kPaged ? (s.page < kBN ? kBN / s.page : 1) : 1;  // pages of a tile
        const int held = kPaged ? (w.q.m + s.page - 1) / s.page : 0;
        int base = 0, cur = -1, nxt = -1;
        auto entry = [&](int e) {
          const int i = e + lane;
          return i < held ? s.table[(size_t)w.q.k0 * s.width + i] : -1;
        };
        auto first_page = [&](int j) { return s.page < kBN ? j * per : (int)((long long)j * kBN / s.page); };
        if constexpr (kPaged) {
          base = first_page(w.j0);
          cur = entry(base);
          nxt = entry(base + 32);
        }
        for (int j = w.j0; ok && j < w.j1; ++j) {
          uint32_t words[4] = {~0u, ~0u, ~0u, ~0u};
          // paged: first row within the page, rows of a copy, copies of a chunk that are made; this lane's copy
          int row = 0, rows = 0, there = 0, my_page = -1;
          if constexpr (kPaged) {
            const int e = first_page(j);
            if (e + per > base + 32) {
              base += 32;
              cur = nxt;
              nxt = entry(base + 32);
            }
            row = s.page < kBN ? 0 : (int)((long long)j * kBN % s.page);
            rows = s.page < kBN ? s.page : kBN;
            my_page = __shfl_sync(0xffffffffu, cur, (e + my_part - base) & 31);
            const bool asked = my_part < per && e + my_part < held;  // behind the sequence's end no page is asked for
            const bool good = asked && my_page >= 0 && my_page < s.pages;
            if (!good || my_chunk >= kChunks) my_page = -1;
            there = __popc(__ballot_sync(0xffffffffu, good && my_chunk == 0));
            const uint32_t gone = __ballot_sync(0xffffffffu, asked && !good && my_chunk == 0);  // bit x: part x
            if (gone) {  // their keys have no weight
              if (lane == 0) atomicOr(ctx.status, kStatusBadPage);
              for (int x = 0; x < per; ++x)
                if ((gone >> x) & 1u) {
                  if (rows >= 32) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                      if (32 * y >= x * rows && 32 * y < (x + 1) * rows) words[y] = 0u;
                  } else {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                      if (y == x >> 1) words[y] &= x & 1 ? 0x0000ffffu : 0xffff0000u;
                  }
                }
            }
          }
#pragma unroll
          for (int kind = 0; kind < 2; ++kind, ++n) {  // 0 = K_j, 1 = V_j
            const int slot = n % R;
            const uint32_t use = n / R;
            // (after a failure no further copy: the issuer goes on until it notices)
            if (lane == 0)
              ok = !*reinterpret_cast<volatile int*>(&ctl->abort) &&
                   (use == 0 || wait_or_abort(&ctl->bar_kv_empty[slot], (use - 1) & 1, ctx, ctl));
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            uint8_t* dst = smem + L::kRingOff + slot * L::kTileBytes;
            const CUtensorMap* map = kind == 0 ? &tmK : &tmV;
            const bool drop = (int)n == ctx.drop_load;
            if constexpr (kPaged) {
              if (lane == 0) {
                if (kind == 1)
                  *reinterpret_cast<uint4*>(ctl->words[slot]) = make_uint4(words[0], words[1], words[2], words[3]);
                if (!drop) {
                  if (there) mbar_arrive_expect_tx(&ctl->bar_kv_full[slot], there * rows * 128 * kChunks);
                  else mbar_arrive(&ctl->bar_kv_full[slot]);
                }
              }
              __syncwarp();
              // a lane a copy
              if (!drop && my_page >= 0)
                tma_load_4d(dst + my_chunk * kChunkBytes + my_part * rows * 128, map, &ctl->bar_kv_full[slot], my_chunk * 64,
                            h, row, my_page);
              if (!drop) kv_armed[slot] = use + 1;
            } else if (lane == 0 && !drop) {
              mbar_arrive_expect_tx(&ctl->bar_kv_full[slot], L::kTileBytes);
#pragma unroll
              for (int c = 0; c < kChunks; ++c)
                tma_load_4d(dst + c * kChunkBytes, map, &ctl->bar_kv_full[slot], c * 64, h, w.q.k0 + j * kBN, 0);
              kv_armed[slot] = use + 1;
            }
          }
        }
      }
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the schedule and computes the descriptors, one elected lane waits and issues.
      uint32_t el_lane;
      const bool el = elect_one_sync(&el_lane);
      bool ok = true;
      uint32_t base = 0;  // ring counter of the item's first K
      uint32_t ne = 0;    // items with at least one key tile
      auto ring_addr = [&](uint32_t n) { return sbase + L::kRingOff + (n % R) * L::kTileBytes; };
      auto wait_el = [&](uint64_t* bar, uint32_t parity) {
        bool r = true;
        if (el) r = wait_or_abort(bar, parity, ctx, ctl);
        return __shfl_sync(0xffffffffu, r ? 1 : 0, el_lane) != 0;
      };
      auto wait_kv = [&](uint32_t n) { return wait_el(&ctl->bar_kv_full[n % R], (n / R) & 1); };
      uint32_t kept_k = 0, kept_v = 0;  // the item's last K and V: their slots are the epilogue's, which releases them
      auto release = [&](uint32_t n) {
        if (el && n != kept_k && n != kept_v) mma_commit(&ctl->bar_kv_empty[n % R]);
      };
      auto issue_s = [&](int t, int qt, uint32_t nk) {
        const uint64_t a0 = sdesc_sw128(sbase + L::kQ + qt * L::kTileBytes, 16, 1024);
        const uint64_t b0 = sdesc_sw128(ring_addr(nk), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
          const uint64_t x = desc_add(a0, off), y = desc_add(b0, off);
          if (el) mma_ss_checked(mg, tmem + (uint32_t)(t * kBN), x, y, kIdescS, kk > 0, kBN);
        }
        if (el) mma_commit(&ctl->bar_s_full[t]);
      };
      auto issue_pv = [&](int t, uint32_t nv, bool acc) {
        const uint64_t b0 = sdesc_sw128(ring_addr(nv), kChunkBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) {
          const uint64_t y = desc_add(b0, kk * 2048);
          if (el)
            mma_ts_checked(mg, tmem + 256 + (uint32_t)(t * D), tmem + (uint32_t)(t * kBN) + kk * 8, y, kIdescPV,
                           (acc || kk > 0) ? 1u : 0u, D);
        }
        if (el) mma_commit(&ctl->bar_pv_done[t]);
      };
      Walk<Pairs> w(share);
      while (w.next(a)) {
        const Item it = item_of(a, w);
        const int c = it.c;
        if (c == 0) continue;
        // After a failure anywhere in the CTA this warp stops issuing but still meets the softmax warps at every
        // named barrier of the schedule.
        if (ok && *reinterpret_cast<volatile int*>(&ctl->abort)) ok = false;
        const int stride = it.split ? 2 : 1;
        kept_k = base + 2 * stage_k(it);
        kept_v = it.split ? kept_k : base + 2 * c - 1;
        int left = it.n[0] + it.n[1];  // products S of this item that are still to come; behind the last the Q tiles are free
        auto last_s = [&] {
          if (--left == 0 && el) mma_commit(&ctl->bar_q_empty);
        };
        auto off = [&](int t, int i) { return (uint32_t)(it.split ? 2 * i + t : i); };  // key tile of slot t's step i
        if (ok) ok = wait_el(&ctl->bar_q_full, ne & 1);
        if (ok) ok = wait_kv(base);
        if (ok) {
          tc_fence_after();
          if (it.n[0] > 0) {
            issue_s(0, 0, base);
            last_s();
          }
          if (it.split) release(base);
          if (el) mma_issued = true;
        }
        if (it.n[1] > 0) {
          if (ok && it.split) ok = wait_kv(base + 2);
          if (ok) {
            tc_fence_after();
            issue_s(1, it.split ? 0 : 1, base + 2 * off(1, 0));
            last_s();
            release(base + 2 * off(1, 0));
          }
        }
        const int steps = max(it.n[0], it.n[1]);
        for (int i = 0; i < steps; ++i) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (i >= it.n[t]) continue;
            const uint32_t nk = base + 2 * off(t, i), nv = nk + 1, nk1 = nk + 2 * stride;
            // V has landed, and, where the slots share their keys, so has the next K: the relay warp waited
            named_sync(kBarP + t, kBarPCount);
            if (ok && i == 0 && ne > 0)  // the previous item's epilogue must have read O before the first P V overwrites it
              ok = wait_el(&ctl->bar_o_free, (ne - 1) & 1);
            if (ok) {
              tc_fence_after();
              issue_pv(t, nv, i > 0);
              if (it.split || t == 1) release(nv);
            }
            if (i + 1 < it.n[t]) {
              if (ok && it.split) ok = wait_kv(nk1);
              if (ok) {
                if (it.split) tc_fence_after();
                issue_s(t, it.split ? 0 : t, nk1);
                last_s();
                if (it.split || t == 1) release(nk1);
              }
            }
            __syncwarp();
          }
        }
        base += 2 * c;
        ++ne;
      }
    } else if (warp >= kRelayWarp) {
      // ------------------------------------------------------------ relay warps
      // All waits for copies and products on behalf of slot t's softmax warps, which wait on named barriers only: a test of
      // an mbarrier takes 150 to 300 cycles beside the matrix instructions' shared-memory reads, even when it passes, and a
      // named barrier about 30.  This warp also looks at V where P V could meet what it must not, tells the softmax warps
      // what the next item is, and sends their rows out.  After a failure it keeps meeting the others.
      const int t = warp - kRelayWarp;
      bool ok = true;
      uint32_t base = 0, g[2] = {0, 0}, ne = 0;  // ring counter; steps of the slots; items with a key tile
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (ok) ok = __all_sync(0xffffffffu, wait_or_abort(bar, phase & 1, ctx, ctl));
      };
      Walk<Pairs> w(share);
      Item it{};
      int par = 0;
      auto post = [&](bool more) {
        Job* job = jobs + 2 * t + par;
        if (lane == 0) {
          if (!more) {
            job->c = -1;
          } else {
            const int tok0 = (2 * w.at.p + (it.split ? 0 : t)) * a.TT;
            job->c = it.c;
            job->n = it.n[t];
            job->j0 = w.j0;
            job->lo = it.lo;
            job->hi = it.hi;
            job->flags = (it.split ? kSplit : 0) | (w.part ? kPart : 0) | (it.split && it.n[1] > 0 ? kJoin : 0) |
                         (tok0 + a.TT <= w.q.n ? kFull : 0);
            job->base = base;
            job->stage = (t == 0 ? base + 2 * stage_k(it) : base + 2 * it.c - 1) % R;
            job->tok0 = tok0;
            job->h = w.at.h;
            job->q = w.q;
            job->ne = ne + 1;
          }
        }
        __syncwarp();
        par ^= 1;
      };
      bool more = w.next(a);
      if (more) it = item_of(a, w);
      post(more);
      named_sync(kBarI + t, kBarRelay);
      while (more) {
        const int c = it.c;
        if (c > 0) {
          // V of step i: an infinity or a NaN in a row of V that not every row of the item reads becomes a zero, and the
          // epilogue adds it to the rows that read it (dirty).  Slot 0 does it where the slots share V, since its product
          // comes first.
          auto look = [&](int i) {
            const uint32_t o = it.split ? 2 * i + t : i, nv = base + 2 * o + 1;
            const int j = w.j0 + (int)o;
            if (!ok || (!it.split && t == 1 && i < it.n[0])) return;
            uint4 words = make_uint4(~0u, ~0u, ~0u, ~0u);
            if constexpr (kPaged) words = *reinterpret_cast<const uint4*>(ctl->words[nv % R]);
            const bool whole = !kPaged || (words.x & words.y & words.z & words.w) == ~0u;
            if (whole && (j + 1) * kBN <= it.lo) return;
            bool bad = false;
#pragma unroll 1
            for (int wr = whole ? max(0, it.lo - j * kBN) & ~31 : 0; wr < kBN; wr += 32) {
              uint4* v = reinterpret_cast<uint4*>(smem + L::kRingOff + (nv % R) * L::kTileBytes + wr * 128) + lane;
              uint4 y[8 * kChunks];
#pragma unroll
              for (int x = 0; x < 8 * kChunks; ++x) y[x] = v[(x / 8) * (kChunkBytes / 16) + (x % 8) * 32];
              uint32_t sum = 0;  // 0 as long as all are finite: an infinity or a NaN times 0 is a NaN
#pragma unroll
              for (int x = 0; x < 8 * kChunks; ++x) {
                sum = times0_plus<kHalf>(y[x].z, times0_plus<kHalf>(y[x].w, sum));
                sum = times0_plus<kHalf>(y[x].x, times0_plus<kHalf>(y[x].y, sum));
              }
              if (!__any_sync(0xffffffffu, not_finite<kHalf>(sum))) continue;
              const uint32_t mw = wr < 64 ? (wr < 32 ? words.x : words.y) : (wr < 96 ? words.z : words.w);
#pragma unroll 1
              for (int x = 0; x < 8 * kChunks; ++x) {
                const int r = 4 * (x % 8) + (lane >> 3), key = j * kBN + wr + r;
                uint4* p = v + (x / 8) * (kChunkBytes / 16) + (x % 8) * 32;
                const uint4 z = *p;
                if (key < it.lo && ((mw >> r) & 1u)) continue;  // every row reads it
                if (!not_finite<kHalf>(z.x) && !not_finite<kHalf>(z.y) && !not_finite<kHalf>(z.z) && !not_finite<kHalf>(z.w))
                  continue;
                bad = true;
                *p = make_uint4(finite_part<kHalf>(z.x), finite_part<kHalf>(z.y), finite_part<kHalf>(z.z),
                                finite_part<kHalf>(z.w));
              }
            }
            if (bad) *reinterpret_cast<volatile uint32_t*>(&ctl->dirty[(ne + 1) & 1]) = ne + 1;
            fence_proxy_async_smem();
            __syncwarp();
          };
          auto nv_of = [&](int i) { return base + 2 * (uint32_t)(it.split ? 2 * i + t : i) + 1; };
          int looked = -1;
          for (int i = 0; i < it.n[t]; ++i) {
            const uint32_t nv = nv_of(i);
            if (looked < i) {
              wait(&ctl->bar_kv_full[nv % R], nv / R);
              look(i);
            }
            wait(&ctl->bar_s_full[t], g[t] + i);
            named_arrive(kBarF + t, kBarRelay);
            looked = i;
            if (i + 1 < it.n[t]) {
              // the next V while the softmax warps are at work, if it is there; and the next K, where the slots share their
              // keys (else the issuer waits for it: this V is not to wait for that K)
              const uint32_t nv1 = nv_of(i + 1);
              if (ok && __all_sync(0xffffffffu, mbar_test(&ctl->bar_kv_full[nv1 % R], (nv1 / R) & 1))) {
                look(i + 1);
                looked = i + 1;
              }
              if (!it.split) wait(&ctl->bar_kv_full[(nv + 1) % R], (nv + 1) / R);
            }
            // A rendezvous: so the softmax warps, whose next step waits for this warp, cannot come to this barrier again
            // before the issuer has passed it, whatever failed.
            named_sync(kBarP + t, kBarPCount);
          }
          // O is complete.  A slot without a step waits for the other's: it must not run ahead, into phases of its barriers
          // that look like others.
          if (it.n[t] > 0) wait(&ctl->bar_pv_done[t], g[t] + it.n[t] - 1);
          if (it.n[t] == 0 || (t == 0 && it.split && it.n[1] > 0)) wait(&ctl->bar_pv_done[1 - t], g[1 - t] + it.n[1 - t] - 1);
          named_arrive(kBarF + t, kBarRelay);
        }
        // where this item's rows go, for the copy below
        const bool out = c > 0 && (t == 0 || !it.split);
        const uint32_t stage = (t == 0 ? base + 2 * stage_k(it) : base + 2 * c - 1) % R;
        const int tok0 = (2 * w.at.p + (it.split ? 0 : t)) * a.TT, h = w.at.h, token = w.q.q0 + tok0;
        const bool full = !w.part && tok0 + a.TT <= w.q.n;
        if (c > 0) {
          g[0] += it.n[0];
          g[1] += it.n[1];
          base += 2 * c;
          ++ne;
        }
        more = w.next(a);
        if (more) it = item_of(a, w);
        post(more);
        if (out) {
          named_sync(kBarOut + t, kBarRelay);
          if (lane == 0 && ok && full && guard_store(ctx, ((size_t)token * s.Hq + h * a.g) * D, D, o_extent)) {
#pragma unroll
            for (int x = 0; x < kChunks; ++x)
              tma_store_4d(smem + L::kRingOff + stage * L::kTileBytes + x * kChunkBytes, &tmO, x * 64, 0, h, token);
            bulk_commit_group();
          }
          __syncwarp();
        }
        named_sync(kBarI + t, kBarRelay);
        if (out && lane == 0) {
          bulk_wait_read_all();
          if (ok) mbar_arrive(&ctl->bar_kv_empty[stage]);
        }
        __syncwarp();
      }
    }
  } else {
    take_registers();
    // ------------------------------------------------------------ softmax warps
    const int t = warp >> 2;                 // slot
    const int row = (warp & 3) * 32 + lane;  // TMEM lane = row of the tile
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t colS = (uint32_t)(t * kBN);
    const int rt = row / a.g, rh = row - rt * a.g;  // token within the tile and head of the group
    const bool in_tile = rt < a.TT;
    if (s.rest) clear_rest(s.starts, s.B, s.T, s.out, (long long)s.Hq * D, s.lse, s.Hq, threadIdx.x, 256);
    for (int par = 0;; par ^= 1) {
      named_sync(kBarI + t, kBarRelay);
      const Job job = jobs[2 * t + par];
      if (job.c < 0) break;
      const bool split = job.flags & kSplit, part = job.flags & kPart, join = job.flags & kJoin;
      const int hq = job.h * a.g + rh, tok = job.tok0 + rt;
      const bool valid = in_tile && tok < job.q.n;
      const int lim = valid ? keys_of(s, job.q, tok) : 0;
      const uint32_t orow = (uint32_t)(job.q.q0 + (valid ? tok : 0)) * s.Hq + hq;  // row of out
      const size_t lo = (size_t)hq * s.T + job.q.q0 + (valid ? tok : 0);
      const bool mine = valid && !(split && t == 1);  // this thread writes the row
      const bool store = mine && guard_store(ctx, (size_t)orow * D, D, o_extent) && guard_store(ctx, lo, 1, lse_extent);
      if (job.c == 0) {  // no key: O = 0 and LSE = -inf, without products or barriers
        if (store) {
#pragma unroll 1
          for (int x = 0; x < D / 8; ++x)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.out) + (size_t)orow * D)[x] = make_uint4(0u, 0u, 0u, 0u);
          s.lse[lo] = -INFINITY;
        }
        continue;
      }
      const int nt = job.n;
      const bool busy = __any_sync(0xffffffffu, valid);  // warps without a row only keep the barriers
      float mu = -INFINITY;  // log2-domain offset in use (scaled maximum, possibly stale by < 2^8)
      float l_run = 0.f;
      for (int i = 0; i < nt; ++i) {
        const int o = split ? 2 * i + t : i, k0 = (job.j0 + o) * kBN;
        named_sync(kBarF + t, kBarRelay);  // S is complete and V has landed
        tc_fence_after();
        if (busy) {
          uint4 words = make_uint4(~0u, ~0u, ~0u, ~0u);
          if constexpr (kPaged) words = *reinterpret_cast<const uint4*>(ctl->words[(job.base + 2 * o + 1) % R]);
          float x[kBN];
          tmem_ld32x2(tl + colS, tl + colS + 32, *reinterpret_cast<float(*)[64]>(&x[0]));
          tmem_ld32x2(tl + colS + 64, tl + colS + 96, *reinterpret_cast<float(*)[64]>(&x[64]));
          const int left = lim - k0;  // lane 0's row, the warp's first, reads the fewest keys
          if (__shfl_sync(0xffffffffu, left, 0) < kBN) {
#pragma unroll
            for (int e = 0; e < kBN; ++e)
              if (e >= left) x[e] = -INFINITY;
          }
          if (kPaged && (words.x & words.y & words.z & words.w) != ~0u) {
            const uint32_t mw[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
            for (int e = 0; e < kBN; ++e)
              if (!((mw[e >> 5] >> (e & 31)) & 1u)) x[e] = -INFINITY;
          }
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = fmaxf(x[e], x[e + 8]);
#pragma unroll
          for (int f = 16; f < kBN; f += 16)
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = max3(m8[e], x[f + e], x[f + e + 8]);
          const float mt = fmaxf(max3(m8[0], m8[1], m8[2]), max3(max3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
          // -inf if the row reads no key of the tile.  The offset stays finite: a score of +inf then gives P = l = +inf,
          // so LSE = +inf and, times 1/l = 0, a row of NaN; a NaN score, which a maximum passes over, gives P = l = NaN.
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
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 y = fma2(make_float2(x[64 * hh + 2 * e], x[64 * hh + 2 * e + 1]), c2, nm2);
              const float2 z = make_float2(ex2(y.x), ex2(y.y));
              rs2 = add2(rs2, z);
              pk[e] = pack2<kHalf>(z.x, z.y);
            }
            tmem_st32_bits(tl + colS + 32 * hh, pk);  // P over the first 64 columns of S
          }
          l_run = l_run * alpha + (rs2.x + rs2.y);
          // P V of the step before, which reads the columns just overwritten and adds to O, is done: it was issued
          // before S, and the commit behind s_full covers every earlier product
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int e = 0; e < D / 32; ++e) {
              float y[32];
              tmem_ld32(tl + 256 + t * D + 32 * e, y);
#pragma unroll
              for (int f = 0; f < 32; ++f) y[f] *= alpha;
              tmem_st32(tl + 256 + t * D + 32 * e, y);
            }
          }
        }
        tc_fence_before();
        named_arrive(kBarP + t, kBarPCount);
      }
      float f0 = 1.f, f1 = 0.f;
      named_sync(kBarF + t, kBarRelay);  // O is complete: this slot's, and for slot 0 of a joined item both
      dbg_late(ctx);
      if (join) {
        // slot 1's rows go to the threads of slot 0, which own the same TMEM lanes; the readers of the sums before these
        // are through, since this item's first P V waited for them
        if (t == 1) {
          sStat[row] = mu;
          sStat[128 + row] = l_run;
        }
        named_sync(kBarL, 256);
        if (t == 0) {
          const float mu1 = sStat[row], top = fmaxf(mu, mu1);
          f0 = mu == -INFINITY ? 0.f : ex2(mu - top);
          f1 = mu1 == -INFINITY ? 0.f : ex2(mu1 - top);
          // (a row of NaN scores has a sum of NaN beside any offset)
          l_run = l_run * f0 + sStat[128 + row] * f1;
          mu = top;
        }
      }
      tc_fence_after();
      if (split && t == 1) {
        tc_fence_before();
        mbar_arrive(&ctl->bar_o_free);
        continue;
      }
      // The way out: 16-bit rows in the slot's free ring slot, 16-byte pieces swizzled as a tensor copy takes them.  A
      // tile of full rows leaves by one; of others this warp stores its 32 rows, D / 8 lanes a row.
      constexpr int kPieces = D / 8;
      uint8_t* out_rows = smem + L::kRingOff + job.stage * L::kTileBytes + (warp & 3) * 32 * 128;
      auto piece = [&](int r, int i) {
        return reinterpret_cast<uint4*>(out_rows + (i >> 3) * kChunkBytes + r * 128 + ((i ^ r) & 7) * 16);
      };
      if (busy) {
        const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
        const bool dirty = *reinterpret_cast<volatile uint32_t*>(&ctl->dirty[job.ne & 1]) == job.ne;
        const int slot = part_of(cta, job.j0);
        if (!join && !dirty && !part) {  // the usual way, 64 columns at a time
#pragma unroll 1
          for (int e = 0; e < D / 64; ++e) {
            float y[64];
            tmem_ld32x2(tl + 256 + t * D + 64 * e, tl + 256 + t * D + 64 * e + 32, y);
#pragma unroll
            for (int f = 0; f < 8; ++f) *piece(lane, 8 * e + f) = pack8<kHalf>(&y[8 * f], inv);
          }
        } else {
#pragma unroll 1
          for (int e = 0; e < D / 32; ++e) {
            float y[32];
            tmem_ld32(tl + 256 + t * D + 32 * e, y);
            if (join) {
              float z[32];
              tmem_ld32(tl + 256 + D + 32 * e, z);
#pragma unroll
              for (int f = 0; f < 32; ++f) y[f] = y[f] * f0 + z[f] * f1;
            }
            if (dirty && valid) {
#pragma unroll 1
              for (int k = max(job.lo, job.j0 * kBN); k < min(lim, (job.j0 + job.c) * kBN); ++k) {
                const uint16_t* v = value_row<kPaged>(a, job.q, job.h, k);
                if (!v) continue;
#pragma unroll
                for (int f = 0; f < 32; ++f) {
                  const float z = load16(v, 32 * e + f, kHalf);
                  if (!isfinite(z)) y[f] += z;
                }
              }
            }
            if (part) {
              float* po = part_o<D>(parts, slot) + t * 128 + row;
              if (valid)
#pragma unroll
                for (int f = 0; f < 32; ++f) po[(size_t)(32 * e + f) * parts.rows] = y[f];
            } else {
#pragma unroll
              for (int f = 0; f < 4; ++f) *piece(lane, 4 * e + f) = pack8<kHalf>(&y[8 * f], inv);
            }
          }
        }
        if (!part && !(job.flags & kFull)) {
          __syncwarp();
          const int some = __popc(__ballot_sync(0xffffffffu, valid));  // rows of tokens that are there come first
#pragma unroll 2
          for (int x = 0; x * (32 / kPieces) < some; ++x) {
            const int r = x * (32 / kPieces) + lane / kPieces;
            const bool to = __shfl_sync(0xffffffffu, store ? 1 : 0, r);
            const uint32_t at = __shfl_sync(0xffffffffu, orow, r);
            if (to)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(s.out) + (size_t)at * D + 8 * (lane % kPieces)) =
                  *piece(r, lane % kPieces);
          }
        }
      }
      fence_proxy_async_smem();
      named_arrive(kBarOut + t, kBarRelay);
      tc_fence_before();
      mbar_arrive(&ctl->bar_o_free);
      if (part) {
        if (valid) part_stat(parts, part_of(cta, job.j0))[t * 128 + row] = make_float2(mu, l_run);
      } else if (store) {
        s.lse[lo] = l_run == 0.f ? -INFINITY : mu * kLn2 + logf(l_run);
      }
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
    if (q_armed) settle(&ctl->bar_q_full, (q_armed - 1) & 1, ctx);
    for (int i = 0; i < R; ++i)
      if (kv_armed[i]) settle(&ctl->bar_kv_full[i], (kv_armed[i] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Joins the parts of the items that were cut.  Block (c - 1, x, y): the item that CTA c's share begins inside of, if no
// earlier share does, rows 32 x .. 32 x + 31, columns 64 y .. 64 y + 63: a lane a row, a warp 8 columns, four parts' loads
// in flight together (one part at a time, all columns: 60 us for one token over 16000 keys by 125 parts, now 31 with the
// attention itself).
template <int D, bool kPaged, bool kHalf>
__global__ void __launch_bounds__(256, 4) seq_join_kernel(const __grid_constant__ SeqArgs a, const Parts parts, int ctas,
                                                          DevCtx ctx) {
  constexpr float kLn2 = 0.6931471805599453f;
  constexpr int kCols = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uaa_seqs& s = a.s;
  const int c = blockIdx.x + 1;
  if (!leads(parts.first, c, s.B)) return;
  const Cut me = parts.first[c];
  const Seq q = load_seq<kPaged>(s, me.b);
  const int lane = threadIdx.x & 31, r = blockIdx.y * 32 + lane, col = blockIdx.z * 64 + (threadIdx.x >> 5) * kCols;
  const int t = r >> 7, rt = (r & 127) / a.g, rh = (r & 127) - rt * a.g;
  const int tok = (2 * me.p + t) * a.TT + rt;
  const bool valid = rt < a.TT && tok < q.n;
  if (!__any_sync(0xffffffffu, valid)) return;
  const int nt = Pairs::inner(a, q, me.p);
  float top = -INFINITY, sum = 0.f, acc[kCols];
#pragma unroll
  for (int x = 0; x < kCols; ++x) acc[x] = 0.f;
  const int at = valid ? r : 0;
  each_part(parts.first, c, ctas, nt, [&](const int (&ids)[kBatch]) {
    float2 st[kBatch];
    float o[kBatch][kCols];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (ids[u] < 0) continue;
      st[u] = part_stat(parts, ids[u])[at];
#pragma unroll
      for (int x = 0; x < kCols; ++x) o[u][x] = part_o<D>(parts, ids[u])[(size_t)(col + x) * parts.rows + at];
    }
    const float before = top;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (ids[u] >= 0) top = fmaxf(top, st[u].x);
    if (before != -INFINITY && top != before) {
      const float f = ex2(before - top);
      sum *= f;
#pragma unroll
      for (int x = 0; x < kCols; ++x) acc[x] *= f;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (ids[u] < 0) continue;
      const float f = st[u].x == -INFINITY ? 0.f : ex2(st[u].x - top);
      sum += st[u].y * f;
#pragma unroll
      for (int x = 0; x < kCols; ++x) acc[x] += o[u][x] * f;
    }
  });
  if (!valid) return;
  const int hq = me.h * a.g + rh;
  const size_t oo = ((size_t)(q.q0 + tok) * s.Hq + hq) * D + col, lo = (size_t)hq * s.T + q.q0 + tok;
  if (!guard_store(ctx, oo, kCols, (size_t)s.T * s.Hq * D) || !guard_store(ctx, lo, 1, (size_t)s.Hq * s.T)) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = static_cast<uint16_t*>(s.out) + oo;
  *reinterpret_cast<uint4*>(out) = pack8<kHalf>(acc, inv);
  if (col == 0) s.lse[lo] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
}

// ---------------------------------------------------------------------------
// Host
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t workspace_bytes(int B, int T, int g, int D, Parts* parts = nullptr, void* at = nullptr) {
  const size_t ctas = device_sms(), rows = part_rows((long long)T * g);
  const size_t first = round256(ctas * sizeof(Cut)), seqs = round256((B + ctas) * sizeof(Seq));
  const size_t o = round256(2 * ctas * rows * D * 4);
  if (parts) {
    char* p = static_cast<char*>(at);
    *parts = Parts{reinterpret_cast<Cut*>(p), reinterpret_cast<Seq*>(p + first),
                   reinterpret_cast<float*>(p + first + seqs), reinterpret_cast<float2*>(p + first + seqs + o), (int)rows};
  }
  return first + seqs + o + round256(2 * ctas * rows * 8);
}

template <int D, bool kPaged, bool kHalf>
int launch(const char* fn, const SeqArgs& a, const Parts& parts, cudaStream_t stream) {
  const uaa_seqs& s = a.s;
  CUtensorMap mq, mk, mv, mo;
  int st;
  const int box = kPaged && s.page < kBN ? s.page : kBN;
  // no key at all: maps of one row over q, which no tile reads
  const bool keys = kPaged ? s.pages > 0 && s.width > 0 : s.Tk > 0;
  const void *k = keys ? s.k : s.q, *v = keys ? s.v : s.q;
  const long long rows = !keys ? 1 : kPaged ? s.page : s.Tk, pages = kPaged && keys ? s.pages : 1;
  const long long kp = kPaged ? s.k_page : s.k_row, vp = kPaged ? s.v_page : s.v_row;
  if ((st = encode_map(&mq, fn, s.q, {D, a.g, s.Hk, s.T}, {s.q_head, a.g * s.q_head, s.q_row}, {64, a.g, 1, a.TT})) ||
      (st = encode_map(&mo, fn, s.out, {D, a.g, s.Hk, s.T}, {D, a.g * D, (long long)s.Hq * D}, {64, a.g, 1, a.TT})) ||
      (st = encode_map(&mk, fn, k, {D, s.Hk, rows, pages}, {s.k_head, s.k_row, kp}, {64, 1, box, 1})) ||
      (st = encode_map(&mv, fn, v, {D, s.Hk, rows, pages}, {s.v_head, s.v_row, vp}, {64, 1, box, 1})))
    return st;
  DevCtx ctx;
  if ((st = get_dev_ctx(&ctx))) return st;
  auto kern = seq_fwd_kernel<D, kPaged, kHalf>;
  const int smem = FwdLayout<D>::kSmem, ctas = device_sms();
  static std::atomic<bool> checked{false};
  cudaError_t e;
  if (!checked.load(std::memory_order_relaxed)) {
    cudaFuncAttributes f{};
    if ((e = cudaFuncGetAttributes(&f, kern)) != cudaSuccess)
      return set_error(UAA_ERR_CUDA, "%s: kernel attributes: %s", fn, cudaGetErrorString(e));
    if (f.numRegs != kLaunchRegs)
      return set_error(UAA_ERR_CUDA, "%s: built with %d registers a thread, not %d", fn, f.numRegs, kLaunchRegs);
    checked.store(true, std::memory_order_relaxed);
  }
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: smem attribute: %s", fn, cudaGetErrorString(e));
  kern<<<ctas, kThreads, smem, stream>>>(mq, mk, mv, mo, a, parts, s.scale * kLog2e, ctx);
  if ((st = check_launch(fn))) return st;
  // items of so few key tiles are not cut
  const long long most = kPaged ? (long long)s.width * s.page : s.Tk;
  if (most <= (2 * kLeastTiles - 1) * kBN) return UAA_OK;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas - 1), (unsigned)(parts.rows / 32), D / 64);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, seq_join_kernel<D, kPaged, kHalf>, a, parts, ctas, ctx);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return check_launch(fn);
}

template <bool kPaged>
int seq_fwd(const char* fn, const uaa_seqs* s, void* workspace, size_t bytes, cudaStream_t stream) {
  int st = check_seqs(fn, s, kPaged);
  if (st) return st;
  if (s->T == 0 || (s->B == 0 && !s->rest)) return UAA_OK;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  const SeqArgs a = seq_args(*s);
  Parts parts;
  const size_t need = workspace_bytes(s->B, s->T, a.g, s->D, &parts, workspace);
  if (bytes < need) return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, bytes, need);
  const bool half = s->dtype == UAA_FP16;
  auto go = s->D == 64 ? (half ? launch<64, kPaged, true> : launch<64, kPaged, false>)
                       : (half ? launch<128, kPaged, true> : launch<128, kPaged, false>);
  return go(fn, a, parts, stream);
}

}  // namespace
}  // namespace uaa

extern "C" size_t uaa_attn_seqs_workspace_bytes(int B, int T, int Hq, int Hk, int D) {
  if (B < 0 || T < 0 || Hk < 1 || Hq < 1 || Hq % Hk || (D != 64 && D != 128)) return 0;
  return uaa::workspace_bytes(B, T, Hq / Hk, D);
}

extern "C" int uaa_attn_packed_fwd(const uaa_seqs* args, void* workspace, size_t workspace_bytes, uaa_stream_t stream) {
  return uaa::seq_fwd<false>("uaa_attn_packed_fwd", args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int uaa_attn_paged_fwd(const uaa_seqs* args, void* workspace, size_t workspace_bytes, uaa_stream_t stream) {
  return uaa::seq_fwd<true>("uaa_attn_paged_fwd", args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
