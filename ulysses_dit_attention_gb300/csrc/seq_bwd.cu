// Attention over packed sequences, backward (the formulas and the row of items that
// is shared out stand in seq_shared.cuh).  No atomics: the same bits every time.
//  1. seq_stats_kernel: Delta = rowsum(dO * O) and -L log2(e) of every row, in tiles
//     of 128 rows as the others read them (row r of a tile: head r % g of token r / g).
//  2. seq_dq_kernel: an item is a tile of query rows; it walks the key tiles that the
//     rows read, with Q and dO in TMEM: S, dP, dQ += dS K.  Rows that read one key tile
//     only get Delta = sum P dP, without the roundings of P and O (with many keys Delta
//     is small beside dP, and so is what they make of it).
//  3. seq_dkdv_kernel: an item is a tile of 128 keys of one sequence and key head; it
//     walks the tiles of query rows that read it:
//        S^T = K Q^T,  P^T = exp2(S^T c - L log2 e),  dP^T = V dO^T,
//        dS^T = P^T (dP^T - Delta),  dV += P^T dO,  dK += dS^T Q   (in TMEM)
//     S and dP once more.  The rows of the g query heads that share the key head are
//     rows of one tile, so their gradients add up in the accumulator.
//  4. seq_bwd_join_kernel: items that were cut between two shares.
// Seven products where five would do; the alternative, dQ by 32-bit reductions from
// the dK/dV kernel, is slower and has no fixed order.
//
// A tile's rows that belong to no token of the sequence are zeros in shared memory
// (those behind a sequence's end would be the next one's): P and dS are 0 there, and
// 0 times what another sequence holds has to be 0.
//
// Bound and times (GB300, on the device).  Long sequences: the chain S, exponentials,
// dP, dS and the products that read them, through TMEM and barriers, one tile at a
// time a CTA: 8192 x 8192, 24 heads, D = 128: 1990 us, by the seven products 1450
// TFLOP/s; 8191 tokens, 24 / 8 heads, causal: dK/dV 541 us (a step 1.65 us for 1.1 us
// of products), dQ 470.  The matrix pipe is active for 58 % (dK/dV) and 45 % (dQ) on
// texts of 326 to 4100 tokens (224 + 215 us).  Short sequences: filling and draining,
// an item costs 5.5 steps beside its own: images of 300 to 1100 tokens, D = 64, 24
// heads: 124 + 96 us at 20 %.  The rows' statistics: memory, 22 us for 108 MB.
#include <math.h>

#include <type_traits>

#include "seq_shared.cuh"

namespace uaa {
namespace {

constexpr int kChunkBytes = 128 * 128;
constexpr int kComputeThreads = 256;  // warps 0-7: TMEM lane quadrant = warp % 4, column half = warp / 4
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kMmaWarp1 = 10;  // the dQ kernel's second issuer
constexpr int kDkdvThreads = 320, kDqThreads = 352;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Packed bf16 pairs of 64 consecutive columns -> 32 TMEM columns.
__device__ __forceinline__ void store_packed64(uint32_t taddr, const float (&x)[64]) {
  uint32_t pk[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) pk[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
  tmem_st32_bits(taddr, pk);
}
// TMEM column of the A operand for K step kk when each half of the 128 columns lies packed at its own half's start.
__device__ __forceinline__ uint32_t packed_a_col(int kk) { return kk < 4 ? kk * 8 : 64 + (kk - 4) * 8; }

// The way out of a gradient tile: this thread's half row (columns hf D / 2 ..) in 16-bit pieces, swizzled as a tensor copy
// takes them.  A tile whose rows all exist leaves by one; of others each warp stores its 32 half rows, a row by D / 16 lanes.
template <int D>
__device__ __forceinline__ uint4* out_piece(uint8_t* tile, int row, int hf, int i) {
  const int p = hf * (D / 16) + i;
  return reinterpret_cast<uint4*>(tile + (p >> 3) * kChunkBytes + row * 128 + (((p ^ row) & 7) << 4));
}
template <int D>
__device__ __forceinline__ void put_columns(uint8_t* tile, int row, int hf, int i0, const float (&v)[32], float f) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *out_piece<D>(tile, row, hf, i0 + e) =
        make_uint4(pack_bf16(v[8 * e + 0] * f, v[8 * e + 1] * f), pack_bf16(v[8 * e + 2] * f, v[8 * e + 3] * f),
                   pack_bf16(v[8 * e + 4] * f, v[8 * e + 5] * f), pack_bf16(v[8 * e + 6] * f, v[8 * e + 7] * f));
}
// to: the offset of this thread's half row in `out`, or ~0 where it is not stored
template <int D>
__device__ __forceinline__ void store_rows(uint8_t* tile, int row0, int hf, __nv_bfloat16* out, size_t to) {
  constexpr int G = D / 16, kRows = 32 / G;  // lanes of a half row, half rows of a store
  const int lane = threadIdx.x & 31;
  __syncwarp();
#pragma unroll 2
  for (int x = 0; x < G; ++x) {
    const int r = x * kRows + lane / G;
    const size_t at = __shfl_sync(0xffffffffu, to, r);
    if (at != ~(size_t)0) *reinterpret_cast<uint4*>(out + at + 8 * (lane % G)) = *out_piece<D>(tile, row0 + r, hf, lane % G);
  }
}

__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void await_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Workspace: per key head and slot of 128 rows Delta and -L log2(e); for each of the two kernels the shares' first places,
// their sequences where they are many, and the parts, (columns, rows) in 32 bits.
struct BwdWork {
  float *delta, *nl2;  // (Hk, slots, 128)
  int slots;
  Cut *first_kv, *first_q;
  Seq *seqs_kv, *seqs_q;
  float *part_kv, *part_q;  // 2 parts a CTA: (2 D, 128): dV then dK; (D, 128)
};
// The first slot of sequence b: sequences do not share slots, and all fit in T / TT + B + 1.
__host__ __device__ __forceinline__ int slots_of(int T, int TT, int B) { return T / TT + B + 1; }
__device__ __forceinline__ int first_slot(const SeqArgs& a, int q0, int b) { return q0 / a.TT + b; }

struct BwdArgs {
  SeqArgs a;
  const __nv_bfloat16* dout;
  __nv_bfloat16 *dq, *dk, *dv;
  BwdWork w;
};

// ---------------------------------------------------------------------------
// 1. A block takes a slot and a key head, eight lanes a row.
template <int D>
__global__ void __launch_bounds__(256) seq_stats_kernel(const __grid_constant__ BwdArgs x) {
  const SeqArgs& a = x.a;
  const uaa_seqs& s = a.s;
  allow_next();
  if (s.B == 0) return;
  const int slot = blockIdx.x, hk = blockIdx.y;
  int lo = 0, hi = s.B - 1;  // the last b whose first slot is not behind this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(a, held_in(s.starts[mid], 0, s.T), mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const Seq q = load_seq<false>(s, lo);
  const int tok0 = (slot - first_slot(a, q.q0, lo)) * a.TT;
  if (tok0 < 0 || tok0 >= q.n) return;
  const size_t to = ((size_t)hk * x.w.slots + slot) * 128;
  const int sub = threadIdx.x & 7;
#pragma unroll
  for (int r0 = 0; r0 < 128; r0 += 32) {
    const int r = r0 + (threadIdx.x >> 3), rt = r / a.g, rh = r - rt * a.g, tok = tok0 + rt;
    const bool valid = rt < a.TT && tok < q.n;
    const int h = hk * a.g + rh;
    const size_t at = ((size_t)(q.q0 + (valid ? tok : 0)) * s.Hq + (valid ? h : 0)) * D;
    const uint4* o = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(s.out) + at);
    const uint4* d = reinterpret_cast<const uint4*>(x.dout + at);
    float acc = 0.f;
    if (valid) {
#pragma unroll
      for (int t = 0; t < D / 64; ++t) {
        const uint4 u = __ldg(o + sub + 8 * t), v = __ldg(d + sub + 8 * t);
        const __nv_bfloat162* u2 = reinterpret_cast<const __nv_bfloat162*>(&u);
        const __nv_bfloat162* v2 = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 uf = __bfloat1622float2(u2[e]), vf = __bfloat1622float2(v2[e]);
          acc = fmaf(uf.x, vf.x, acc);
          acc = fmaf(uf.y, vf.y, acc);
        }
      }
    }
    acc += __shfl_xor_sync(0xffffffffu, acc, 4);
    acc += __shfl_xor_sync(0xffffffffu, acc, 2);
    acc += __shfl_xor_sync(0xffffffffu, acc, 1);
    if (sub == 0) {
      const float l = valid ? s.lse[(size_t)h * s.T + q.q0 + tok] : -INFINITY;
      x.w.delta[to + r] = acc;
      // a row without a key, or none: P = 0; where a score was NaN or +inf: P = NaN
      x.w.nl2[to + r] = l == -INFINITY ? -INFINITY : l < INFINITY ? -l * kLog2e : NAN;
    }
  }
}

// ---------------------------------------------------------------------------
// 3. dK / dV
template <int D>
struct DkdvLayout {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTileBytes;
  static constexpr int kQStages = 3;  // Q_i (+ Delta_i): last read by dK_i
  static constexpr int kDStages = 2;  // dO_i (+ -L log2 e): last read by dV_i
  static constexpr int kQ = kV + kTileBytes;
  static constexpr int kDO = kQ + kQStages * kTileBytes;
  static constexpr int kLse = kDO + kDStages * kTileBytes;
  static constexpr int kDelta = kLse + kDStages * 128 * 4;
  static constexpr int kCtl = kDelta + kQStages * 128 * 4;  // find_share's scratch lies over kLse .. kCtl
  static constexpr int kKept = kCtl + 256;
  static constexpr int kSeqs = D == 128 ? 16 : kKeptSeqs;  // as many as there is room for
  static constexpr int kSmem = kKept + kSeqs * 16;
  static_assert(kSmem <= 232448, "dK/dV shared memory exceeds the per-CTA limit");
};

struct DkdvCtl {
  uint64_t bar_kv_full, bar_kv_empty;
  uint64_t bar_q_full[3], bar_q_empty[3];
  uint64_t bar_do_full[2], bar_do_empty[2];
  uint64_t bar_s_full, bar_dp_full, bar_p_ready, bar_ds_ready;
  uint64_t bar_acc_done, bar_acc_free, bar_final, bar_tail, bar_out;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DkdvCtl) <= 256, "control block");

// Zeros in rows from .. to - 1 of a tile (a warp), for the async proxy to read.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int to, int lane) {
  for (int i = lane; i < (to - from) * (D / 8); i += 32) {
    const int r = from + i / (D / 8), c = i % (D / 8);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * kChunkBytes + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kDkdvThreads, 1)
    seq_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const __grid_constant__ CUtensorMap tmDK, const __grid_constant__ CUtensorMap tmDV,
                    const __grid_constant__ BwdArgs x, float scale_log2, DevCtx ctx) {
  using L = DkdvLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr uint32_t kIdescKK = idesc_bf16_f32(128, 128, false, false);  // S^T, dP^T
  constexpr uint32_t kIdescKM = idesc_bf16_f32(128, D, false, true);     // dV, dK (A in TMEM)
  constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;

  extern __shared__ __align__(1024) uint8_t smem[];
  DkdvCtl* ctl = reinterpret_cast<DkdvCtl*>(smem + L::kCtl);
  float* sLse = reinterpret_cast<float*>(smem + L::kLse);
  float* sDelta = reinterpret_cast<float*>(smem + L::kDelta);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    // the swizzled operand tiles need 1024-byte alignment; never expected to trigger
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const SeqArgs& a = x.a;
  const uaa_seqs& s = a.s;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rows = a.TT * a.g;  // of a query tile

  if (threadIdx.x == 0) {
    // a Q_i / dO_i stage is read by two products, each releasing it by a commit
    mbar_init(&ctl->bar_kv_full, 1);
    mbar_init(&ctl->bar_kv_empty, 1);
    for (int i = 0; i < L::kQStages; ++i) {
      mbar_init(&ctl->bar_q_full[i], 1);
      mbar_init(&ctl->bar_q_empty[i], 2);
    }
    for (int i = 0; i < L::kDStages; ++i) {
      mbar_init(&ctl->bar_do_full[i], 1);
      mbar_init(&ctl->bar_do_empty[i], 2);
    }
    mbar_init(&ctl->bar_s_full, 1);
    mbar_init(&ctl->bar_dp_full, 1);
    mbar_init(&ctl->bar_p_ready, kComputeThreads);
    mbar_init(&ctl->bar_ds_ready, kComputeThreads);
    mbar_init(&ctl->bar_acc_done, 1);
    mbar_init(&ctl->bar_acc_free, kComputeThreads);
    mbar_init(&ctl->bar_final, 1);
    mbar_init(&ctl->bar_tail, 1);
    mbar_init(&ctl->bar_out, kComputeThreads);
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
  // rows of a query tile that no copy fills (and, at an item's end, that its way out has been through)
  if (rows < 128 && warp < L::kQStages + L::kDStages)
    zero_rows<D>(smem + L::kQ + warp * L::kTileBytes, rows, 128, lane);
  const Share share = find_share<KeyRow, false, kDkdvThreads, L::kSeqs>(a, smem + L::kLse, smem + L::kKept, x.w.seqs_kv,
                                                                       ctx.status);
  fence_proxy_async_smem();  // its scratch is where copies will land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) x.w.first_kv[blockIdx.x] = share.from;
  await_previous();  // the rows' statistics, and the dQ kernel's corrections of them
  allow_next();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t k_extent = (size_t)s.Tk * s.Hk * D;

  uint32_t q_armed[3] = {0, 0, 0}, do_armed[2] = {0, 0}, kv_armed = 0, tails = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t nq = 0, it = 0;
    Walk<KeyRow> w(share);
    while (ok && w.next(a)) {
      if (w.j1 <= w.j0) continue;
      const int hk = w.at.h;
      if (lane == 0) {
        if (it > 0) ok = wait_or_abort(&ctl->bar_kv_empty, (it - 1) & 1, ctx, ctl);
        if (ok) {
          mbar_arrive_expect_tx(&ctl->bar_kv_full, 2 * L::kTileBytes);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kK + c * kChunkBytes, &tmK, &ctl->bar_kv_full, c * 64, hk, w.q.k0 + w.at.p * kBN, 0);
            tma_load_4d(smem + L::kV + c * kChunkBytes, &tmV, &ctl->bar_kv_full, c * 64, hk, w.q.k0 + w.at.p * kBN, 0);
          }
          kv_armed = it + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      const int lt0 = KeyRow::first(a, w.q, w.at.p), slot0 = first_slot(a, w.q.q0, w.at.b);
      for (int i = w.j0; ok && i < w.j1; ++i, ++nq) {
        const int lt = lt0 + i, tok0 = lt * a.TT;
        const int left = held_in(w.q.n - tok0, 0, a.TT) * a.g;  // the tile's rows that belong to the sequence
        const size_t stats = ((size_t)hk * x.w.slots + slot0 + lt) * 128;
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {  // Q_i with its Delta row, then dO_i with its -L log2(e) row
          const int st = kind == 0 ? nq % L::kQStages : nq % L::kDStages;
          const uint32_t use = kind == 0 ? nq / L::kQStages : nq / L::kDStages;
          uint64_t* full = kind == 0 ? &ctl->bar_q_full[st] : &ctl->bar_do_full[st];
          uint64_t* empty = kind == 0 ? &ctl->bar_q_empty[st] : &ctl->bar_do_empty[st];
          uint8_t* dst = smem + (kind == 0 ? L::kQ : L::kDO) + st * L::kTileBytes;
          if (lane == 0 && use > 0) ok = wait_or_abort(empty, (use - 1) & 1, ctx, ctl);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (kind == 0 && (int)nq == ctx.drop_load) continue;
          // The last tile's other rows are the next sequence's: it lands on a barrier of its own, they become zeros, and
          // then it is full.
          uint64_t* land = left < rows ? &ctl->bar_tail : full;
          if (lane == 0) {
            mbar_arrive_expect_tx(land, rows * 128 * kChunks + 512);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(dst + c * kChunkBytes, kind == 0 ? &tmQ : &tmDO, land, c * 64, 0, hk, w.q.q0 + tok0);
            bulk_load(kind == 0 ? sDelta + st * 128 : sLse + st * 128, (kind == 0 ? x.w.delta : x.w.nl2) + stats, 512, land);
          }
          if (left < rows) {
            ++tails;
            bool r = true;
            if (lane == 0) r = wait_or_abort(land, (tails - 1) & 1, ctx, ctl);
            ok = __shfl_sync(0xffffffffu, r, 0);
            if (!ok) break;
            zero_rows<D>(dst, left, rows, lane);
            if (lane == 0) mbar_arrive(full);
          }
          if (kind == 0) q_armed[st] = use + 1;
          else do_armed[st] = use + 1;
        }
      }
      ++it;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    // One elected lane issues the four products of every query tile i in the order
    //   S^T_0 dP^T_0 | dV_0 S^T_1 | dK_0 dP^T_1 | dV_1 S^T_2 | dK_1 dP^T_2 | ...
    // each burst after the compute warps' handshake that it depends on: dV_i and S^T_{i+1} after p_ready(i) (the compute
    // warps arrive only once Q_{i+1} has landed), dK_i and dP^T_{i+1} after ds_ready(i) (dO_{i+1} landed).  The products
    // of one thread run in order: dV_i reads P^T_i before S^T_{i+1} overwrites those columns, dK_i reads dS^T_i before
    // dP^T_{i+1} does.
    uint32_t el_lane;
    const bool el = elect_one_sync(&el_lane);
    bool ok = true;
    uint32_t nq = 0, it = 0;
    auto sq = [&](uint32_t g) { return sbase + L::kQ + (g % L::kQStages) * L::kTileBytes; };
    auto sdo = [&](uint32_t g) { return sbase + L::kDO + (g % L::kDStages) * L::kTileBytes; };
    auto wait_el = [&](uint64_t* bar, uint32_t parity) {
      bool r = true;
      if (el) r = wait_or_abort(bar, parity, ctx, ctl);
      return __shfl_sync(0xffffffffu, r ? 1 : 0, el_lane) != 0;
    };
    // S^T_g = K Q_g^T (c = 0) or dP^T_g = V dO_g^T (c = 1)
    auto issue_kk = [&](int c, uint32_t g) {
      const uint64_t a0 = sdesc_sw128(sbase + (c == 0 ? L::kK : L::kV), 16, 1024);
      const uint64_t b0 = sdesc_sw128(c == 0 ? sq(g) : sdo(g), 16, 1024);
      const uint32_t d = tmem + (c == 0 ? kColS : kColDP);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
        const uint64_t y = desc_add(a0, off), z = desc_add(b0, off);
        if (el) mma_ss_checked(mg, d, y, z, kIdescKK, kk > 0, 128);
      }
      if (el) {
        mma_commit(c == 0 ? &ctl->bar_s_full : &ctl->bar_dp_full);
        mma_commit(c == 0 ? &ctl->bar_q_empty[g % L::kQStages] : &ctl->bar_do_empty[g % L::kDStages]);
      }
    };
    // dV += P^T dO_g (c = 0) or dK += dS^T Q_g (c = 1)
    // (the last Q and dO of an item stay: their stages are the epilogue's, which releases them)
    auto issue_acc = [&](int c, uint32_t g, bool first, bool last) {
      const uint64_t b0 = sdesc_sw128(c == 0 ? sdo(g) : sq(g), kChunkBytes, 1024);
      const uint32_t d = tmem + (c == 0 ? kColDV : kColDK);
      const uint32_t p = tmem + (c == 0 ? kColS : kColDP);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint64_t z = desc_add(b0, kk * 2048);
        if (el) mma_ts_checked(mg, d, p + packed_a_col(kk), z, kIdescKM, (!first || kk > 0) ? 1u : 0u, D);
      }
      if (el && !last) mma_commit(c == 0 ? &ctl->bar_do_empty[g % L::kDStages] : &ctl->bar_q_empty[g % L::kQStages]);
    };
    // behind the last product that reads K or V
    auto release_kv = [&] {
      if (el) mma_commit(&ctl->bar_kv_empty);
    };
    Walk<KeyRow> w(share);
    while (ok && w.next(a)) {
      const int nt = w.j1 - w.j0;
      if (nt <= 0) continue;
      ok = wait_el(&ctl->bar_kv_full, it & 1);
      if (ok) ok = wait_el(&ctl->bar_q_full[nq % L::kQStages], (nq / L::kQStages) & 1);
      if (ok) ok = wait_el(&ctl->bar_do_full[nq % L::kDStages], (nq / L::kDStages) & 1);
      if (ok) {
        tc_fence_after();
        issue_kk(0, nq);
        issue_kk(1, nq);
        if (nt == 1) release_kv();
        if (el) mma_issued = true;
      }
      for (int i = 0; ok && i < nt; ++i) {
        const uint32_t g = nq + i;
        const bool more = i + 1 < nt;
        if (!(ok = wait_el(&ctl->bar_p_ready, g & 1))) break;
        if (i == 0 && it > 0) {
          // the previous item's epilogue must have read dK / dV
          if (!(ok = wait_el(&ctl->bar_acc_free, (it - 1) & 1))) break;
        }
        tc_fence_after();
        issue_acc(0, g, i == 0, !more);
        if (more) issue_kk(0, g + 1);
        if (!(ok = wait_el(&ctl->bar_ds_ready, g & 1))) break;
        tc_fence_after();
        issue_acc(1, g, i == 0, !more);
        if (more) issue_kk(1, g + 1);
        if (i + 2 == nt) release_kv();
      }
      if (el) {
        if (ok) {
          mma_commit(&ctl->bar_acc_done);
        } else {
          *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
        }
      }
      __syncwarp();
      nq += nt;
      ++it;
    }
  } else {
    // ------------------------------------------------------------ compute warps 0..7
    const int quad = warp & 3;
    const int hf = warp >> 2;
    const int jrow = quad * 32 + lane;  // key = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    bool ok = true;
    uint32_t nq = 0, it = 0;
    if (s.rest) {
      const int* starts = s.starts_k ? s.starts_k : s.starts;
      clear_rest(starts, s.B, s.Tk, x.dk, (long long)s.Hk * D, nullptr, 0, threadIdx.x, kComputeThreads);
      clear_rest(starts, s.B, s.Tk, x.dv, (long long)s.Hk * D, nullptr, 0, threadIdx.x, kComputeThreads);
    }
    Walk<KeyRow> w(share);
    while (ok && w.next(a)) {
      const int nt = w.j1 - w.j0, key = w.at.p * kBN + jrow;
      const bool there = key < w.q.m;
      const size_t off = ((size_t)(w.q.k0 + (there ? key : 0)) * s.Hk + w.at.h) * D + hf * (D / 2);
      const bool store = there && guard_store(ctx, off, D / 2, k_extent);  // this thread's half row of dK, dV
      if (nt <= 0) {  // no query reads this tile: dK = dV = 0
        if (store && !w.part) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            *reinterpret_cast<uint4*>(x.dk + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(x.dv + off + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        continue;
      }
      // the first row of query tile lt that reads this key: (key - (m - n) - lt TT) g
      const int lt0 = KeyRow::first(a, w.q, w.at.p) + w.j0, reach = key - (w.q.m - w.q.n);
      for (int i = 0; i < nt; ++i) {
        const uint32_t g = nq + i;
        const int qs = g % L::kQStages;
        const int ds = g % L::kDStages;
        // -L log2(e) of the tile lies with dO, Delta with Q; both have landed before S^T is complete
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_do_full[ds], (g / L::kDStages) & 1, ctx, ctl));
        if (!ok) break;
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_q_full[qs], (g / L::kQStages) & 1, ctx, ctl));
        if (!ok) break;
        if (i + 1 < nt) {
          const uint32_t g1 = g + 1;  // Q_{i+1}, read by the S^T that this tile's p_ready releases
          ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_q_full[g1 % L::kQStages], (g1 / L::kQStages) & 1, ctx, ctl));
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_s_full, g & 1, ctx, ctl));
        if (!ok) break;
        tc_fence_after();
        float p[64];
        tmem_ld32x2(tl + kColS + 64 * hf, tl + kColS + 64 * hf + 32, p);
        {
          const float2* nl2 = reinterpret_cast<const float2*>(sLse + ds * 128 + 64 * hf);
          const float2 c2 = make_float2(scale_log2, scale_log2);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 y = fma2(make_float2(p[2 * c], p[2 * c + 1]), c2, nl2[c]);
            p[2 * c] = ex2(y.x);
            p[2 * c + 1] = ex2(y.y);
          }
          if (s.causal) {  // rows that do not read this key
            const int from = held_in(reach - (lt0 + i) * a.TT, 0, 128) * a.g - 64 * hf;
            if (__any_sync(0xffffffffu, from > 0)) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (c < from) p[c] = 0.f;
            }
          }
        }
        // P^T as bf16 over the first 32 columns of this half's S^T
        store_packed64(tl + kColS + 64 * hf, p);
        tc_fence_before();
        mbar_arrive(&ctl->bar_p_ready);
        if (i + 1 < nt) {
          const uint32_t g1 = g + 1;  // dO_{i+1}, read by the dP^T that this tile's ds_ready releases
          ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_do_full[g1 % L::kDStages], (g1 / L::kDStages) & 1, ctx, ctl));
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dp_full, g & 1, ctx, ctl));
        if (!ok) break;
        tc_fence_after();
        float dp[64];
        tmem_ld32x2(tl + kColDP + 64 * hf, tl + kColDP + 64 * hf + 32, dp);
        {
          const float2* dl = reinterpret_cast<const float2*>(sDelta + qs * 128 + 64 * hf);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 d = mul2(make_float2(p[2 * c], p[2 * c + 1]), sub2(make_float2(dp[2 * c], dp[2 * c + 1]), dl[c]));
            dp[2 * c] = d.x;
            dp[2 * c + 1] = d.y;
          }
        }
        store_packed64(tl + kColDP + 64 * hf, dp);
        tc_fence_before();
        mbar_arrive(&ctl->bar_ds_ready);
      }
      if (!ok) break;
      // epilogue: dV, and dK = scale (dS^T Q)
      ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_acc_done, it & 1, ctx, ctl));
      if (!ok) break;
      tc_fence_after();
      float* part = x.w.part_kv + (size_t)part_of(blockIdx.x, w.j0) * (2 * D * 128) + jrow;
      const uint32_t gl = nq + nt - 1;  // dK leaves through the last Q's stage, dV through the last dO's
      uint8_t* out[2] = {smem + L::kDO + (gl % L::kDStages) * L::kTileBytes,
                         smem + L::kQ + (gl % L::kQStages) * L::kTileBytes};
      const bool whole = !w.part && (w.at.p + 1) * kBN <= w.q.m;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {  // 32 columns of dV and of dK in turn
        const int col = hf * (D / 2) + 32 * (c >> 1), which = c & 1;
        float v[32];
        tmem_ld32(tl + (which ? kColDK : kColDV) + col, v);
        if (w.part) {
#pragma unroll
          for (int e = 0; e < 32; ++e) part[(size_t)(which * D + col + e) * 128] = v[e];
        } else {
          put_columns<D>(out[which], jrow, hf, 4 * (c >> 1), v, which ? s.scale : 1.f);
        }
      }
      tc_fence_before();
      mbar_arrive(&ctl->bar_acc_free);
      if (!w.part && !whole) {
        const size_t to = store ? off : ~(size_t)0;
        store_rows<D>(out[0], quad * 32, hf, x.dv, to);
        store_rows<D>(out[1], quad * 32, hf, x.dk, to);
      }
      fence_proxy_async_smem();
      mbar_arrive(&ctl->bar_out);
      if (warp == 0) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_out, it & 1, ctx, ctl));
        if (!ok) break;
        if (lane == 0) {
          if (whole && store) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              tma_store_4d(out[0] + c * kChunkBytes, &tmDV, c * 64, w.at.h, w.q.k0 + w.at.p * kBN, 0);
              tma_store_4d(out[1] + c * kChunkBytes, &tmDK, c * 64, w.at.h, w.q.k0 + w.at.p * kBN, 0);
            }
            bulk_commit_group();
            bulk_wait_read_all();
          }
        }
        __syncwarp();
        // dV and dK were put in all rows of the two tiles.  Those that no copy fills are zeros again before the tiles are a
        // stage again: the next item's products read them, and an infinity or a NaN there would reach all of its rows.
        if (rows < 128 && !w.part) {
          zero_rows<D>(out[0], rows, 128, lane);
          zero_rows<D>(out[1], rows, 128, lane);
        }
        if (lane == 0) {
          mbar_arrive(&ctl->bar_do_empty[gl % L::kDStages]);
          mbar_arrive(&ctl->bar_q_empty[gl % L::kQStages]);
        }
        __syncwarp();
      }
      nq += nt;
      ++it;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp && mma_issued) {
    // every MMA has completed before TMEM is released (mma_issued: the issuing lane)
    mma_commit(&ctl->bar_final);
    settle(&ctl->bar_final, 0, ctx);
  }
  if (warp == kProducerWarp && lane == 0) {
    if (kv_armed) settle(&ctl->bar_kv_full, (kv_armed - 1) & 1, ctx);
    if (tails) settle(&ctl->bar_tail, (tails - 1) & 1, ctx);
    for (int i = 0; i < 3; ++i)
      if (q_armed[i]) settle(&ctl->bar_q_full[i], (q_armed[i] - 1) & 1, ctx);
    for (int i = 0; i < 2; ++i)
      if (do_armed[i]) settle(&ctl->bar_do_full[i], (do_armed[i] - 1) & 1, ctx);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// 2. dQ
template <int D>
struct DqLayout {
  // K and V in rings of their own: a K slot is freed only by dQ, late in a key tile's processing, a V slot already by dP.
  // Behind them an item's Q and dO, on their way into TMEM.
  static constexpr int kKRing = (D == 128) ? 3 : 6;
  static constexpr int kVRing = (D == 128) ? 2 : 5;
  static constexpr int kRing = kKRing + kVRing;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kQ = kRing * kTileBytes;
  static constexpr int kDO = kQ + kTileBytes;
  static constexpr int kCtl = kDO + kTileBytes;
  static constexpr int kKept = kCtl + 512;
  static constexpr int kSeqs = D == 128 ? 32 : kKeptSeqs;  // as many as there is room for
  static constexpr int kSums = kKept + kSeqs * 16;  // of the rows' two halves; find_share's scratch before
  static constexpr int kSmem = kSums + 2 * 128 * 8;
  static_assert(kShareBytes <= 2 * 128 * 8, "scratch");
  static_assert(kSmem <= 232448, "dQ shared memory exceeds the per-CTA limit");
};

struct DqCtl {
  uint64_t bar_qdo_ready;
  uint64_t bar_kv_full[16], bar_kv_empty[16];
  uint64_t bar_s_full, bar_s_read, bar_dp_full, bar_ds_ready;
  uint64_t bar_dq_done, bar_dq_free, bar_final[2], bar_dq_step, bar_tail, bar_out, bar_qd_full, bar_qd_free,
      bar_sums;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DqCtl) <= 512, "control block");

using Rows = QueryRow<1>;
// What a row's P may add up to beside one: the error of its scores and of lse.
constexpr float kNearOne = 1.f / 1024;

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
    seq_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ BwdArgs x, float scale_log2, DevCtx ctx) {
  using L = DqLayout<D>;
  constexpr int kChunks = D / 64;
  constexpr int R = L::kRing;
  constexpr int KR = L::kKRing, VR = L::kVRing;
  auto kslot = [](uint32_t g) { return (int)(g % KR); };
  auto vslot = [](uint32_t g) { return KR + (int)(g % VR); };
  auto kpar = [](uint32_t g) { return (g / KR) & 1u; };
  auto vpar = [](uint32_t g) { return (g / VR) & 1u; };
  constexpr uint32_t kIdescKK = idesc_bf16_f32(128, 128, false, false);  // S, dP
  constexpr uint32_t kIdescKM = idesc_bf16_f32(128, D, false, true);     // dQ (A in TMEM)
  // TMEM: S, dP (then dS), the dQ accumulator, and Q / dO as A operands of S / dP
  constexpr uint32_t kColS = 0, kColDP = 128, kColDQ = 256, kColQ = 384, kColDO = 448;

  extern __shared__ __align__(1024) uint8_t smem[];
  DqCtl* ctl = reinterpret_cast<DqCtl*>(smem + L::kCtl);
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) atomicOr(ctx.status, kStatusBadLaunch);
    return;
  }
  const SeqArgs& a = x.a;
  const uaa_seqs& s = a.s;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->bar_qdo_ready, kComputeThreads);
    for (int i = 0; i < R; ++i) {
      mbar_init(&ctl->bar_kv_full[i], 1);
      mbar_init(&ctl->bar_kv_empty[i], i < KR ? 2 : 1);  // K: S and dQ read it; V: dP only
    }
    mbar_init(&ctl->bar_s_full, 1);
    // the compute warps plus the other issuer's hand-over (see the issuers)
    mbar_init(&ctl->bar_s_read, kComputeThreads + 1);
    mbar_init(&ctl->bar_dp_full, 1);
    mbar_init(&ctl->bar_ds_ready, kComputeThreads + 1);
    mbar_init(&ctl->bar_dq_done, 1);
    mbar_init(&ctl->bar_dq_free, kComputeThreads);
    mbar_init(&ctl->bar_dq_step, 1);
    mbar_init(&ctl->bar_tail, 1);
    mbar_init(&ctl->bar_out, kComputeThreads);
    mbar_init(&ctl->bar_qd_full, 1);
    mbar_init(&ctl->bar_qd_free, kComputeThreads);
    mbar_init(&ctl->bar_sums, kComputeThreads);
    mbar_init(&ctl->bar_final[0], 1);
    mbar_init(&ctl->bar_final[1], 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmDO);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  const Share share = find_share<Rows, false, kDqThreads, L::kSeqs>(a, smem + L::kSums, smem + L::kKept, x.w.seqs_q,
                                                                    ctx.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) x.w.first_q[blockIdx.x] = share.from;
  allow_next();
  const uint32_t tmem = ctl->tmem_base;
  const MmaGuard mg = mma_guard(ctx, sbase, L::kSmem, tmem, 512);  // debug builds' operand checks
  const size_t q_extent = (size_t)s.T * s.Hq * D;

  uint32_t kv_armed[R] = {}, tails = 0, qd_armed = 0;
  bool mma_issued = false;

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t n = 0, gp = 0, it = 0;  // n: loads, gp: key tiles loaded
    Walk<Rows> w(share);
    while (ok && w.next(a)) {
      if (w.j1 <= w.j0) continue;
      if (lane == 0) {
        if (it > 0) ok = wait_or_abort(&ctl->bar_qd_free, (it - 1) & 1, ctx, ctl);
        if (ok) {
          const int at = w.q.q0 + w.at.p * a.TT;
          mbar_arrive_expect_tx(&ctl->bar_qd_full, 2 * a.TT * a.g * 128 * kChunks);
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tma_load_4d(smem + L::kQ + c * kChunkBytes, &tmQ, &ctl->bar_qd_full, c * 64, 0, w.at.h, at);
            tma_load_4d(smem + L::kDO + c * kChunkBytes, &tmDO, &ctl->bar_qd_full, c * 64, 0, w.at.h, at);
          }
          qd_armed = it + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++it;
      for (int j = w.j0; ok && j < w.j1; ++j, ++gp) {
        const int left = held_in(w.q.m - j * kBN, 0, kBN);  // the tile's keys that belong to the sequence
#pragma unroll
        for (int kind = 0; kind < 2; ++kind, ++n) {  // 0 = K_j, 1 = V_j
          const int slot = kind == 0 ? kslot(gp) : vslot(gp);
          const uint32_t use = kind == 0 ? gp / KR : gp / VR;
          if (lane == 0 && use > 0) ok = wait_or_abort(&ctl->bar_kv_empty[slot], (use - 1) & 1, ctx, ctl);
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if ((int)n == ctx.drop_load) continue;
          // dQ += dS K takes rows of K behind the sequence's end times 0: they become zeros before the slot is full
          const bool tail = kind == 0 && left < kBN;
          uint64_t* land = tail ? &ctl->bar_tail : &ctl->bar_kv_full[slot];
          uint8_t* dst = smem + slot * L::kTileBytes;
          if (lane == 0) {
            mbar_arrive_expect_tx(land, L::kTileBytes);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_load_4d(dst + c * kChunkBytes, kind == 0 ? &tmK : &tmV, land, c * 64, w.at.h, w.q.k0 + j * kBN, 0);
          }
          if (tail) {
            ++tails;
            bool r = true;
            if (lane == 0) r = wait_or_abort(land, (tails - 1) & 1, ctx, ctl);
            ok = __shfl_sync(0xffffffffu, r, 0);
            if (!ok) break;
            zero_rows<D>(dst, left, kBN, lane);
            if (lane == 0) mbar_arrive(&ctl->bar_kv_full[slot]);
          }
          kv_armed[slot] = use + 1;
        }
      }
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp1) {
    // ------------------------------------------------------------ MMA issuers (lane 0 of warps 9 and 10)
    // Two chains, each issued by its own thread, per key tile g:
    //   warp 9  (chain s): S_0 | S_1 | S_2 | ...              (S_{g+1} after s_read(g))
    //   warp 10 (chain d): dP_0 | dQ_0 dP_1 | dQ_1 dP_2 | ... (after ds_ready(g))
    // The threads take turns burst by burst; the turn is handed over through the handshake barriers themselves: chain d
    // arrives on s_read(g) behind dP_g, chain s on ds_ready(g) once it has issued all but four products of S_{g+1} (after
    // the last key tile, once s_read(last) has completed).  dQ_g and dP_{g+1} both take A from TMEM, and such products of
    // one thread are not reliably in order: dP_{g+1} is issued only once dQ_g has completed.
    const int c = warp - kMmaWarp;  // 0: chain s, 1: chain d
    bool ok = true;
    uint32_t g = 0, it = 0;  // key tiles across items; items with one
    uint32_t dq_step = 0;    // chain d: dQ completions waited for
    auto slot_addr = [&](int slot) { return sbase + slot * L::kTileBytes; };
    auto pass_turn = [&]() { mbar_arrive(c == 0 ? &ctl->bar_ds_ready : &ctl->bar_s_read); };
    auto issue_s = [&](uint32_t gg, bool pass) {
      const uint64_t b0 = sdesc_sw128(slot_addr(kslot(gg)), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
        mma_ts_checked(mg, tmem + kColS, tmem + kColQ + kk * 8, desc_add(b0, off), kIdescKK, kk > 0, 128);
        if (pass && kk == (D / 16 > 4 ? D / 16 - 5 : 0)) pass_turn();
      }
      mma_commit(&ctl->bar_s_full);
      mma_commit(&ctl->bar_kv_empty[kslot(gg)]);
    };
    auto issue_dp = [&](uint32_t gg) {
      const uint64_t b0 = sdesc_sw128(slot_addr(vslot(gg)), 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * kChunkBytes + (kk & 3) * 32;
        mma_ts_checked(mg, tmem + kColDP, tmem + kColDO + kk * 8, desc_add(b0, off), kIdescKK, kk > 0, 128);
      }
      pass_turn();
      mma_commit(&ctl->bar_dp_full);
      mma_commit(&ctl->bar_kv_empty[vslot(gg)]);
    };
    // (the last K of an item stays: its slot is the epilogue's, which releases it)
    auto issue_dq = [&](uint32_t gg, bool first, bool last) {
      const uint64_t b0 = sdesc_sw128(slot_addr(kslot(gg)), kChunkBytes, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_checked(mg, tmem + kColDQ, tmem + kColDP + packed_a_col(kk), desc_add(b0, kk * 2048), kIdescKM,
                       (!first || kk > 0) ? 1u : 0u, D);
      if (!last) mma_commit(&ctl->bar_kv_empty[kslot(gg)]);
    };
    Walk<Rows> w(share);
    while (ok && w.next(a)) {
      const int ntl = w.j1 - w.j0;
      if (ntl <= 0) continue;
      if (lane == 0) {
        // Q and dO of this item are in TMEM.  Past the first key tile the compute warps arrive on s_read / ds_ready only
        // after they have seen K / V of the next tile land, so no other wait is needed.
        ok = wait_or_abort(&ctl->bar_qdo_ready, it & 1, ctx, ctl);
        if (ok)
          ok = c == 0 ? wait_or_abort(&ctl->bar_kv_full[kslot(g)], kpar(g), ctx, ctl)
                      : wait_or_abort(&ctl->bar_kv_full[vslot(g)], vpar(g), ctx, ctl);
        if (ok) {
          tc_fence_after();
          if (c == 0) issue_s(g, false);
          else issue_dp(g);
          mma_issued = true;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      for (int i = 0; ok && i < ntl; ++i) {
        const bool more = i + 1 < ntl;
        if (lane == 0) {
          if (c == 0) {
            ok = wait_or_abort(&ctl->bar_s_read, g & 1, ctx, ctl);
            if (ok) {
              tc_fence_after();
              if (more) issue_s(g + 1, true);
              else pass_turn();
            }
          } else {
            ok = wait_or_abort(&ctl->bar_ds_ready, g & 1, ctx, ctl);
            if (ok && i == 0 && it > 0) ok = wait_or_abort(&ctl->bar_dq_free, (it - 1) & 1, ctx, ctl);
            if (ok) {
              tc_fence_after();
              issue_dq(g, i == 0, !more);
              if (more) {
                mma_commit(&ctl->bar_dq_step);
                ok = wait_or_abort(&ctl->bar_dq_step, dq_step & 1, ctx, ctl);
                ++dq_step;
                if (ok) {
                  tc_fence_after();
                  issue_dp(g + 1);
                }
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++g;
      }
      if (!ok) break;
      if (lane == 0 && c == 1) mma_commit(&ctl->bar_dq_done);
      __syncwarp();
      ++it;
    }
    if (!ok && lane == 0) *reinterpret_cast<volatile int*>(&ctl->abort) = 1;  // the other issuer waits for our hand-over
  } else {
    // ------------------------------------------------------------ compute warps 0..7
    const int quad = warp & 3;
    const int hf = warp >> 2;
    const int row = quad * 32 + lane;  // query row = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
    const int rt = row / a.g, rh = row - rt * a.g;
    bool ok = true;
    uint32_t g = 0, it = 0;
    if (s.rest) clear_rest(s.starts, s.B, s.T, x.dq, (long long)s.Hq * D, nullptr, 0, threadIdx.x, kComputeThreads);
    await_previous();  // the rows' statistics
    uint32_t alone = 0;  // items of one key tile
    Walk<Rows> w(share);
    while (ok && w.next(a)) {
      const int tok = w.at.p * a.TT + rt, hq = w.at.h * a.g + rh;
      const bool valid = rt < a.TT && tok < w.q.n;
      const int lim = valid ? keys_of(s, w.q, tok) : 0, lo = keys_of(s, w.q, w.at.p * a.TT);
      const size_t qoff = ((size_t)(w.q.q0 + (valid ? tok : 0)) * s.Hq + (valid ? hq : 0)) * D;
      const bool store = valid && guard_store(ctx, qoff + hf * (D / 2), D / 2, q_extent);  // this thread's half row
      const int ntl = w.j1 - w.j0;
      if (ntl <= 0) {  // no key: dQ = 0
        if (store && !w.part) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            *reinterpret_cast<uint4*>(x.dq + qoff + hf * (D / 2) + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      {
        // Q (hf = 0) or dO from shared memory into TMEM: the previous item's products have all completed (its dq_done was
        // waited for).  Rows of no token become zeros.
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_qd_full, it & 1, ctx, ctl));
        if (!ok) break;
        const uint8_t* src = smem + (hf == 0 ? L::kQ : L::kDO) + row * 128;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t wv[32];
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + c * kChunkBytes + (((t ^ row) & 7) << 4));
            wv[4 * t + 0] = valid ? v.x : 0u;
            wv[4 * t + 1] = valid ? v.y : 0u;
            wv[4 * t + 2] = valid ? v.z : 0u;
            wv[4 * t + 3] = valid ? v.w : 0u;
          }
          tmem_st32_bits(tl + (hf == 0 ? kColQ : kColDO) + 32 * c, wv);
        }
        mbar_arrive(&ctl->bar_qd_free);
        tc_fence_before();
        mbar_arrive(&ctl->bar_qdo_ready);
      }
      auto prow = [&] { return ((size_t)w.at.h * x.w.slots + first_slot(a, w.q.q0, w.at.b) + w.at.p) * 128 + row; };
      const float nl2 = x.w.nl2[prow()];
      float dl = x.w.delta[prow()];
      // A key tile; kAlone: the only one that the rows read (a body of its own: as a branch of the other one images of 300 to
      // 1100 tokens, which have none of these, take 326 us a step instead of 320).
      auto tile = [&](auto only, int i) {
        constexpr bool kAlone = decltype(only)::value;
        const int j = w.j0 + i;
        // K and V of the next tile are read by the products that this tile's s_read and ds_ready release; they normally
        // land long before, and waiting for them here keeps these waits off the issuing threads.
        if (!kAlone && i + 1 < ntl) {
          bool okw = wait_or_abort(&ctl->bar_kv_full[kslot(g + 1)], kpar(g + 1), ctx, ctl);
          if (okw) okw = wait_or_abort(&ctl->bar_kv_full[vslot(g + 1)], vpar(g + 1), ctx, ctl);
          ok = __all_sync(0xffffffffu, okw);
          if (!ok) return;
        }
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_s_full, g & 1, ctx, ctl));
        if (!ok) return;
        tc_fence_after();
        float p[64];
        tmem_ld32x2(tl + kColS + 64 * hf, tl + kColS + 64 * hf + 32, p);
        tc_fence_before();
        mbar_arrive(&ctl->bar_s_read);
        const int left = lim - j * kBN - 64 * hf;  // keys of this half that the row reads
        const bool edge = (j + 1) * kBN > lo;
        {
          const float2 c2 = make_float2(scale_log2, scale_log2);
          const float2 n2 = make_float2(nl2, nl2);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 y = fma2(make_float2(p[2 * c], p[2 * c + 1]), c2, n2);
            p[2 * c] = ex2(y.x);
            p[2 * c + 1] = ex2(y.y);
          }
        }
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dp_full, g & 1, ctx, ctl));
        if (!ok) return;
        tc_fence_after();
        if constexpr (kAlone) {
          // Delta = sum P dP, from both halves of the row, which the dK/dV kernel reads too.  Where few keys are read, what
          // dout . out is off by (the roundings of P and of out) shows in dS: dQ and dK of sequences of 2, 9 and 40 tokens,
          // causal, are off by 0.0037, 0.0030 and 0.0027 with it and by 0.0024 without; of 32 sequences of 60 to 128 tokens
          // a step takes 124 us instead of 120.  (P that do not add up to one are of a call over some of the keys with the
          // lse of all of them, or of a checkpoint: dout . out is their Delta.)
          // A softmax over one key is constant: with P = 1 Delta is dP itself, so dS is 0, here and in the dK/dV kernel, whose dP
          // is the same sum of the same products.
          if (lim == 1 && hf == 0 && fabsf(p[0] - 1.f) < kNearOne) p[0] = 1.f;
          float sum[4] = {}, both[4] = {};  // of every fourth key: short chains
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y[32];
            tmem_ld32(tl + kColDP + 64 * hf + 32 * e, y);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (32 * e + c < left) {
                sum[c & 3] += p[32 * e + c];
                both[c & 3] = fmaf(p[32 * e + c], y[c], both[c & 3]);
              }
          }
          float2* sums = reinterpret_cast<float2*>(smem + L::kSums) + row;
          sums[hf * 128] = make_float2((sum[0] + sum[1]) + (sum[2] + sum[3]), (both[0] + both[1]) + (both[2] + both[3]));
          mbar_arrive(&ctl->bar_sums);
          ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_sums, alone & 1, ctx, ctl));
          if (!ok) return;
          ++alone;
          if (fabsf(sums[0].x + sums[128].x - 1.f) < kNearOne) {
            dl = sums[0].y + sums[128].y;
            if (hf == 0) x.w.delta[prow()] = dl;
          }
        }
        float dp[64];
        tmem_ld32x2(tl + kColDP + 64 * hf, tl + kColDP + 64 * hf + 32, dp);
        {
          const float2 d2 = make_float2(dl, dl);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 d = mul2(make_float2(p[2 * c], p[2 * c + 1]), sub2(make_float2(dp[2 * c], dp[2 * c + 1]), d2));
            dp[2 * c] = d.x;
            dp[2 * c + 1] = d.y;
          }
          if (edge) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c >= left) dp[c] = 0.f;
          }
        }
        store_packed64(tl + kColDP + 64 * hf, dp);
        tc_fence_before();
        mbar_arrive(&ctl->bar_ds_ready);
        ++g;
      };
      if (ntl == 1 && !w.part) {
        tile(std::true_type{}, 0);
      } else {
        for (int i = 0; ok && i < ntl; ++i) tile(std::false_type{}, i);
      }
      if (!ok) break;
      // epilogue: dQ = scale (dS K)
      ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_dq_done, it & 1, ctx, ctl));
      if (!ok) break;
      tc_fence_after();
      float* part = x.w.part_q + (size_t)part_of(blockIdx.x, w.j0) * (D * 128) + row;
      uint8_t* out = smem + kslot(g - 1) * L::kTileBytes;  // dQ leaves through the last K's slot
      const bool whole = !w.part && (w.at.p + 1) * a.TT <= w.q.n;
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        const int col = hf * (D / 2) + 32 * c;
        float v[32];
        tmem_ld32(tl + kColDQ + col, v);
        if (w.part) {
#pragma unroll
          for (int e = 0; e < 32; ++e) part[(size_t)(col + e) * 128] = v[e];
        } else {
          put_columns<D>(out, row, hf, 4 * c, v, s.scale);
        }
      }
      tc_fence_before();
      mbar_arrive(&ctl->bar_dq_free);
      if (!w.part && !whole) store_rows<D>(out, quad * 32, hf, x.dq, store ? qoff + hf * (D / 2) : ~(size_t)0);
      fence_proxy_async_smem();
      mbar_arrive(&ctl->bar_out);
      if (warp == 0) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->bar_out, it & 1, ctx, ctl));
        if (!ok) break;
        if (lane == 0) {
          if (whole && store) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
              tma_store_4d(out + c * kChunkBytes, &tmDQ, c * 64, 0, w.at.h, w.q.q0 + w.at.p * a.TT);
            bulk_commit_group();
            bulk_wait_read_all();
          }
          mbar_arrive(&ctl->bar_kv_empty[kslot(g - 1)]);
        }
        __syncwarp();
      }
      ++it;
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if ((warp == kMmaWarp || warp == kMmaWarp1) && lane == 0 && mma_issued) {
    mma_commit(&ctl->bar_final[warp - kMmaWarp]);
    settle(&ctl->bar_final[warp - kMmaWarp], 0, ctx);
  }
  if (warp == kProducerWarp && lane == 0) {
    if (tails) settle(&ctl->bar_tail, (tails - 1) & 1, ctx);
    if (qd_armed) settle(&ctl->bar_qd_full, (qd_armed - 1) & 1, ctx);
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
// 4. Adds up the parts of the items that were cut, in their order.  Block (c - 1, x, kernel): 32 rows, a lane a row, a
// warp an eighth of the columns; kernel 0: dK and dV, 1: dQ.
template <int D>
__global__ void __launch_bounds__(256) seq_bwd_join_kernel(const __grid_constant__ BwdArgs x, int ctas, DevCtx ctx) {
  await_previous();
  const SeqArgs& a = x.a;
  const uaa_seqs& s = a.s;
  const int c = blockIdx.x + 1, lane = threadIdx.x & 31, r = blockIdx.y * 32 + lane, warp = threadIdx.x >> 5;
  const bool keys = blockIdx.z == 0;
  const Cut* first = keys ? x.w.first_kv : x.w.first_q;
  if (!leads(first, c, s.B)) return;
  const Cut me = first[c];
  const Seq q = load_seq<false>(s, me.b);
  const int nt = keys ? KeyRow::inner(a, q, me.p) : Rows::inner(a, q, me.p);
  const int cols = keys ? D / 4 : D / 8;  // of a warp
  const size_t size = (keys ? 2 : 1) * D * 128;
  const float* part = (keys ? x.w.part_kv : x.w.part_q) + r;
  bool valid;
  size_t off;
  if (keys) {
    const int key = me.p * kBN + r;
    valid = key < q.m;
    off = ((size_t)(q.k0 + (valid ? key : 0)) * s.Hk + me.h) * D;
  } else {
    const int rt = r / a.g, rh = r - rt * a.g, tok = me.p * a.TT + rt;
    valid = rt < a.TT && tok < q.n;
    off = ((size_t)(q.q0 + (valid ? tok : 0)) * s.Hq + me.h * a.g + (valid ? rh : 0)) * D;
  }
#pragma unroll 1
  for (int c0 = warp * cols; c0 < (warp + 1) * cols; c0 += 8) {
    float acc[8] = {};
    each_part(first, c, ctas, nt, [&](const int (&ids)[kBatch]) {
      float v[kBatch][8];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[u][e] = ids[u] < 0 ? 0.f : part[(size_t)ids[u] * size + (size_t)(c0 + e) * 128];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += v[u][e];
    });
    const bool dv = keys && c0 < D;
    const float f = dv ? 1.f : s.scale;
    const int col = keys && !dv ? c0 - D : c0;
    __nv_bfloat16* to = keys ? (dv ? x.dv : x.dk) : x.dq;
    if (valid && guard_store(ctx, off + col, 8, keys ? (size_t)s.Tk * s.Hk * D : (size_t)s.T * s.Hq * D))
      *reinterpret_cast<uint4*>(to + off + col) =
          make_uint4(pack_bf16(acc[0] * f, acc[1] * f), pack_bf16(acc[2] * f, acc[3] * f),
                     pack_bf16(acc[4] * f, acc[5] * f), pack_bf16(acc[6] * f, acc[7] * f));
  }
}

// ---------------------------------------------------------------------------
// Host
size_t bwd_workspace(int B, int T, int Hk, int g, int D, BwdWork* w = nullptr, void* at = nullptr) {
  const size_t ctas = device_sms(), slots = slots_of(T, 128 / g, B);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(at) + used;
    used += (bytes + 255) & ~(size_t)255;
    return static_cast<void*>(p);
  };
  BwdWork x;
  x.slots = (int)slots;
  x.delta = static_cast<float*>(take(Hk * slots * 512));
  x.nl2 = static_cast<float*>(take(Hk * slots * 512));
  x.first_kv = static_cast<Cut*>(take(ctas * sizeof(Cut)));
  x.first_q = static_cast<Cut*>(take(ctas * sizeof(Cut)));
  x.seqs_kv = static_cast<Seq*>(take((B + ctas) * sizeof(Seq)));
  x.seqs_q = static_cast<Seq*>(take((B + ctas) * sizeof(Seq)));
  x.part_kv = static_cast<float*>(take(2 * ctas * 2 * D * 128 * 4));
  x.part_q = static_cast<float*>(take(2 * ctas * D * 128 * 4));
  if (w) *w = x;
  return used;
}

template <typename K, typename... Args>
int launch_after(const char* fn, K kern, dim3 grid, int threads, int smem, cudaStream_t stream, Args... args) {
  cudaError_t e = cudaSuccess;
  if (smem) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: smem attribute: %s", fn, cudaGetErrorString(e));
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return set_error(UAA_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return check_launch(fn);
}

template <int D>
int launch_bwd(const char* fn, const BwdArgs& x, cudaStream_t stream) {
  const uaa_seqs& s = x.a.s;
  const SeqArgs& a = x.a;
  CUtensorMap mq, mk, mv, md, oq, ok, ov;
  int st;
  // without queries, or without keys, the maps lie over the other's tensor and no tile reads them
  const bool some = s.T > 0, keys = s.Tk > 0;
  const void *q = some ? s.q : s.k, *d = some ? static_cast<const void*>(x.dout) : s.k;
  const void *k = keys ? s.k : s.q, *v = keys ? s.v : s.q;
  const long long T = some ? s.T : 1, Tk = keys ? s.Tk : 1;
  if ((st = encode_map(&mq, fn, q, {D, a.g, s.Hk, T}, {s.q_head, a.g * s.q_head, s.q_row}, {64, a.g, 1, a.TT})) ||
      (st = encode_map(&md, fn, d, {D, a.g, s.Hk, T}, {D, a.g * D, (long long)s.Hq * D}, {64, a.g, 1, a.TT})) ||
      (st = encode_map(&oq, fn, some ? x.dq : x.dk, {D, a.g, s.Hk, T}, {D, a.g * D, (long long)s.Hq * D},
                       {64, a.g, 1, a.TT})) ||
      (st = encode_map(&ok, fn, keys ? x.dk : x.dq, {D, s.Hk, Tk, 1}, {D, s.Hk * D, s.Hk * D}, {64, 1, kBN, 1})) ||
      (st = encode_map(&ov, fn, keys ? x.dv : x.dq, {D, s.Hk, Tk, 1}, {D, s.Hk * D, s.Hk * D}, {64, 1, kBN, 1})) ||
      (st = encode_map(&mk, fn, k, {D, s.Hk, Tk, 1}, {s.k_head, s.k_row, s.k_row}, {64, 1, kBN, 1})) ||
      (st = encode_map(&mv, fn, v, {D, s.Hk, Tk, 1}, {s.v_head, s.v_row, s.v_row}, {64, 1, kBN, 1})))
    return st;
  DevCtx ctx;
  if ((st = get_dev_ctx(&ctx))) return st;
  const int ctas = device_sms();
  const float c = s.scale * kLog2e;
  seq_stats_kernel<D><<<dim3(x.w.slots, s.Hk), 256, 0, stream>>>(x);
  if ((st = check_launch(fn))) return st;
  if (some && (st = launch_after(fn, seq_dq_kernel<D>, dim3(ctas), kDqThreads, DqLayout<D>::kSmem, stream, mq, md, mk, mv,
                                 oq, x, c, ctx)))
    return st;
  if ((st = launch_after(fn, seq_dkdv_kernel<D>, dim3(ctas), kDkdvThreads, DkdvLayout<D>::kSmem, stream, mq, mk, mv, md, ok,
                         ov, x, c, ctx)))
    return st;
  if (!some) return UAA_OK;  // nothing was cut: no tile has an inner one
  return launch_after(fn, seq_bwd_join_kernel<D>, dim3(ctas - 1, 4, 2), 256, 0, stream, x, ctas, ctx);
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" size_t uaa_attn_packed_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int D) {
  if (B < 0 || T < 0 || Hk < 1 || Hq < 1 || Hq % Hk || Hq / Hk > 128 || (D != 64 && D != 128)) return 0;
  return bwd_workspace(B, T, Hk, Hq / Hk, D);
}

extern "C" int uaa_attn_packed_bwd(const uaa_seqs* s, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                   size_t workspace_bytes, uaa_stream_t stream) {
  const char* fn = "uaa_attn_packed_bwd";
  int st = check_seqs(fn, s, false, true);
  if (st) return st;
  if (s->dtype != UAA_BF16) return set_error(UAA_ERR_UNSUPPORTED, "%s: the backward is built for bf16", fn);
  if ((s->B == 0 && !s->rest) || (s->T == 0 && s->Tk == 0)) return UAA_OK;
  if (s->T > 0 && ((st = check_dev_ptr(fn, "dout", dout)) || (st = check_dev_ptr(fn, "dq", dq)))) return st;
  if (s->Tk > 0 && ((st = check_dev_ptr(fn, "dk", dk)) || (st = check_dev_ptr(fn, "dv", dv)))) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  BwdArgs x{seq_args(*s), static_cast<const __nv_bfloat16*>(dout), static_cast<__nv_bfloat16*>(dq),
            static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv), {}};
  const size_t need = bwd_workspace(s->B, s->T, s->Hk, x.a.g, s->D, &x.w, workspace);
  if (workspace_bytes < need)
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  if (s->Hk > 65535) return set_error(UAA_ERR_UNSUPPORTED, "%s: Hk must be <= 65535", fn);
  return s->D == 64 ? launch_bwd<64>(fn, x, static_cast<cudaStream_t>(stream))
                    : launch_bwd<128>(fn, x, static_cast<cudaStream_t>(stream));
}
