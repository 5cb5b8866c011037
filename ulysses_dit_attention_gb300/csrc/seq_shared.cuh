// Shared by the kernels of attention over sequences of their own lengths: packed
// one behind the other, or with their keys and values in the pages of a cache.
//
// Sequence b has n queries (tokens starts[b] .. starts[b+1]) and m keys; its last
// query stands at its last key, so with `causal` query i reads keys 0 .. m - n + i,
// without it all of them.  g = Hq / Hk query heads share a key head:
//   S = scale q . k,  P = softmax(S),  O = P V,  L = log sum exp S,
//   Delta = dO . O,  dS = P (dO . V - Delta),
//   dV = sum P dO,  dK = scale sum dS Q  (over the rows of the g heads),  dQ = scale dS K.
//
// The lengths are in device memory, so nothing on the host has seen them: every
// kernel cuts them to what the tensors hold before it uses them.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "uaa_common.cuh"

namespace uaa {

int check_dev_ptr(const char* fn, const char* name, const void* p);

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4-D tiled tensor store from shared memory (bulk-group completion).
__device__ __forceinline__ void tma_store_4d(const void* smem_src, const CUtensorMap* map, int c0, int c1, int c2,
                                             int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// What the row of items depends on.
struct Shape {
  int causal, Hk, TT;
};
struct SeqArgs {
  uaa_seqs s;
  int g;   // query heads of a key head
  int TT;  // tokens of a tile of 128 rows, a row being one head of one token
  __device__ __forceinline__ operator Shape() const { return Shape{s.causal, s.Hk, TT}; }
};

__device__ __forceinline__ int held_in(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// One sequence: its first query token, its queries, its first key token (packed) or table row (paged), its keys.
struct alignas(16) Seq {
  int q0, n, k0, m;
};

// `bad`: its table row or its length lies outside the cache.
template <bool kPaged>
__device__ __forceinline__ Seq load_seq(const uaa_seqs& s, int b, bool* bad = nullptr) {
  Seq r;
  r.q0 = held_in(s.starts[b], 0, s.T);
  r.n = held_in(s.starts[b + 1], r.q0, s.T) - r.q0;
  if constexpr (kPaged) {
    r.k0 = s.seqs ? s.seqs[b] : b;
    const bool there = r.k0 >= 0 && r.k0 < s.table_rows;
    r.k0 = there ? r.k0 : 0;
    const int m = there ? s.lens[r.k0] : -1;
    const long long most = (long long)s.width * s.page;
    if (bad) *bad = m < 0 || m > most;
    r.m = m < 0 ? 0 : (int)min((long long)m, most);
  } else {
    const int* st = s.starts_k ? s.starts_k : s.starts;
    r.k0 = held_in(st[b], 0, s.Tk);
    r.m = held_in(st[b + 1], r.k0, s.Tk) - r.k0;
    if (bad) *bad = false;
  }
  return r;
}

// Keys that query i of the sequence reads.
__device__ __forceinline__ int keys_of(int causal, const Seq& q, int i) {
  return causal ? held_in(q.m - q.n + i + 1, 0, q.m) : q.m;
}
__device__ __forceinline__ int keys_of(const uaa_seqs& s, const Seq& q, int i) { return keys_of(s.causal, q, i); }

// Zeros to the tokens of no sequence, before starts[0] and behind starts[B], of a (T, row) tensor of 16-bit elements: the
// calling threads, `n` of them a block, take 16-byte pieces in turn.  lse: -inf beside them, of `heads` heads.
__device__ __noinline__ void clear_rest(const int* starts, int B, int T, void* x, long long row, float* lse, int heads,
                                        int thread, int n) {
  const int a = held_in(starts[0], 0, T), b = held_in(starts[B], a, T);
  const long long head = (long long)a * row / 8, skip = (long long)(b - a) * row / 8;
  const long long all = head + (long long)(T - b) * row / 8;
  for (long long i = (long long)blockIdx.x * n + thread; i < all; i += (long long)gridDim.x * n)
    static_cast<uint4*>(x)[i < head ? i : i + skip] = make_uint4(0u, 0u, 0u, 0u);
  const long long none = T - (b - a);
  for (long long i = (long long)blockIdx.x * n + thread; lse && i < none * heads; i += (long long)gridDim.x * n) {
    const long long h = i / none, t = i - h * none;
    lse[h * T + (t < a ? t : t + (b - a))] = -INFINITY;
  }
}

__device__ __forceinline__ float load16(const void* p, size_t at, int fp16) {
  return fp16 ? __half2float(static_cast<const __half*>(p)[at]) : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

// ---------------------------------------------------------------------------
// A row of items and its shares.  Each kernel works on tiles (of queries or of keys) of every sequence and key head, and
// an item's inner loop runs over tiles of the other kind; the items of all sequences stand in a row, (sequence, head,
// tile), weighed by the tokens that the inner loop meets plus those that its filling and draining
// cost (`item`), and the row is cut into equal shares, one a CTA,
// in the middle of an item where it falls so.  A kind of row says how many tiles a sequence has, how many inner tiles a
// tile has and what the first p tiles weigh.
constexpr int kBN = 128;  // keys of a tile
constexpr int kMostTokens = 1 << 30;  // of a tensor, or of a sequence's pages: places are 32-bit sums of them and a tile
// The least inner tiles of a part (1: images of 300 to 1100 tokens 94 us instead of 87).  A share may weigh as little as one,
// and an item weighs several, so that small calls have an item or a part a CTA (at least 4: one token over 700 keys 18.4 us
// instead of 16.2 in a graph, prompts of 150, 8 and 10 tokens 15.8 instead of 11.6).
constexpr int kLeastTiles = 2;

__device__ __forceinline__ int tiles_in(int x, int per) { return (x + per - 1) / per; }

// (of a guess that is put right)
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tiles of W query tokens, inner tiles of keys: tile p's last query reads the most keys (the last tile weighs as if it
// were full).  Of a causal sequence with fewer keys than queries the first `none` tiles read no key.
template <int kTilesOf2>  // tiles of 128 rows: 1 or 2 (a pair)
struct QueryRow {
  static __device__ __forceinline__ int width(const Shape& a) { return kTilesOf2 * a.TT; }
  static __device__ __forceinline__ int tiles(const Shape& a, const Seq& q) { return tiles_in(q.n, width(a)); }
  static __device__ __forceinline__ int inner(const Shape& a, const Seq& q, int p) {
    return tiles_in(keys_of(a.causal, q, min(q.n, (p + 1) * width(a)) - 1), kBN);
  }
  static __device__ __forceinline__ int unit(const Shape&) { return kBN; }  // tokens of an inner tile
  // A pair's costs 3 key tiles' time (4.4 us beside 1.44 us at D = 128) and the half tile that is rounded up; a single
  // tile's (dQ) was measured: of 2, 3, 4 and 5 tiles 3 is the fastest or within 1 %.
  static constexpr int item = kTilesOf2 == 2 ? 7 * kBN / 2 : 3 * kBN;
  int none;
  long long flat, slope;  // item none + (P = p - none) flat + slope P (P + 1) / 2
  __device__ __forceinline__ QueryRow(const Shape& a, const Seq& q) {
    const int W = width(a), off = q.m - q.n;
    none = a.causal && off < 0 ? -off / W : 0;
    flat = item + (a.causal ? (long long)off + (long long)none * W : q.m);
    slope = a.causal ? W : 0;
  }
  __device__ __forceinline__ long long of(int p) const {
    const long long P = p - none;
    return P <= 0 ? (long long)item * p : (long long)item * none + P * flat + slope * (P * (P + 1) / 2);
  }
  __device__ __forceinline__ int guess(long long w) const {
    const float x = (float)(w - (long long)item * none);
    if (x <= 0.f) return (int)((float)w * (1.f / item));
    if (!slope) return none + (int)__fdividef(x, (float)flat);
    const float h = 0.5f * (float)slope, f = (float)flat + h;
    return none + (int)__fdividef(2.f * x, f + root(f * f + 4.f * h * x));
  }
};

// Tiles of 128 keys, inner tiles of TT query tokens: min(n, m - 128 p) queries read keys of tile p.
struct KeyRow {
  static __device__ __forceinline__ int tiles(const Shape&, const Seq& q) { return tiles_in(q.m, kBN); }
  static __device__ __forceinline__ int first(const Shape& a, const Seq& q, int p) {  // the first inner tile
    return a.causal ? max(0, p * kBN - (q.m - q.n)) / a.TT : 0;
  }
  static __device__ __forceinline__ int inner(const Shape& a, const Seq& q, int p) {
    return max(0, tiles_in(q.n, a.TT) - first(a, q, p));
  }
  static __device__ __forceinline__ int unit(const Shape& a) { return a.TT; }
  int item;  // (of 1.5 to 8 inner tiles 4 to 7 are the fastest within 2 %)
  int full;  // the first tiles, which all queries read
  long long n, m;
  __device__ __forceinline__ KeyRow(const Shape& a, const Seq& q) : item(11 * a.TT / 2), n(q.n), m(q.m) {
    full = !a.causal ? INT32_MAX : q.m >= q.n ? (q.m - q.n) / kBN + 1 : 0;
  }
  __device__ __forceinline__ long long of(int p) const {
    const long long f = min(p, full), P = p;
    return P * item + f * n + (P - f) * m - kBN / 2 * (P * (P - 1) - f * (f - 1));
  }
  __device__ __forceinline__ int guess(long long w) const {
    const long long f = (long long)full * (item + n);
    const float flat = (float)(item + n);
    if (w <= f) return (int)__fdividef((float)w, flat);
    // behind the full tiles: x = b P - 64 P (P - 1) with P = p - full
    const float x = (float)(w - f), b = (float)(item + m - (long long)kBN * full) + kBN / 2;
    return full + (int)__fdividef(2.f * x, b + root(fmaxf(b * b - 2.f * kBN * x, 0.f)));
  }
};

// A place in the row: inner tile j of tile p of sequence b, key head h.
struct Cut {
  int b, h, p, j;
};
__device__ __forceinline__ bool same_item(const Cut& x, const Cut& y) { return x.b == y.b && x.h == y.h && x.p == y.p; }
__device__ __forceinline__ bool before(const Cut& x, const Cut& y) {  // x's item lies before y's
  return x.b != y.b ? x.b < y.b : x.h != y.h ? x.h < y.h : x.p < y.p;
}
struct Found {  // weight w of sequence b
  Seq q;
  long long w;
  int b;
};

// The place at weight w of a sequence.  (Called from one place: a share's end has to be the next one's beginning.)
template <class Row>
__device__ __forceinline__ Cut cut_at(const Shape& a, const Seq& q, long long w, int b) {
  const int np = Row::tiles(a, q);
  const Row row(a, q);
  const long long head = row.of(np);
  Cut c{b, min((int)__fdividef((float)w, (float)head), a.Hk - 1), 0, 0};
  while (c.h > 0 && c.h * head > w) --c.h;
  while ((c.h + 1) * head <= w) ++c.h;
  w -= c.h * head;
  c.p = held_in(row.guess(w), 0, np - 1);  // the last p with of(p) <= w: guessed in 32 bits, put right
  while (c.p > 0 && row.of(c.p) > w) --c.p;
  while (c.p + 1 < np && row.of(c.p + 1) <= w) ++c.p;
  const long long first = row.of(c.p);
  const int nt = Row::inner(a, q, c.p);
  c.j = min((int)(__fdividef((float)(w - first), (float)(row.of(c.p + 1) - first)) * nt + 0.5f), nt);
  if (c.j < kLeastTiles) {
    c.j = 0;
  } else if (nt - c.j < kLeastTiles) {
    c.j = 0;
    if (++c.p == np) {
      c.p = 0;
      if (++c.h == a.Hk) {
        c.h = 0;
        ++c.b;
      }
    }
  }
  return c;
}

// The share of a CTA, with its sequences as they are now: all roles of the CTA walk it over this copy, so that they agree
// on every item, after a failure and if someone writes into the lengths meanwhile.
constexpr int kKeptSeqs = 64;      // sequences of a share that shared memory usually has room for (more: the workspace)
constexpr int kShareBytes = 512;   // shared scratch of find_share
struct Share {
  Cut from, to;
  const Seq* kept;  // of sequence from.b and the next ones
};
// All threads of the block.  `spill`: kept sequences of all shares, CTA c's from its first sequence + c on.
template <class Row, bool kPaged, int kThreads, int kKept = kKeptSeqs>
__device__ __forceinline__ Share find_share(const SeqArgs& a, uint8_t* scratch, uint8_t* kept_smem, Seq* spill,
                                            unsigned int* status) {
  const uaa_seqs& s = a.s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x, ctas = gridDim.x;
  auto weigh = [&](int b, Seq& q, bool tell) {
    bool bad;
    q = load_seq<kPaged>(s, b, &bad);
    if (bad && tell && cta == 0) atomicOr(status, kStatusBadPage);
    const int np = Row::tiles(a, q);
    return np > 0 ? s.Hk * Row(a, q).of(np) : 0LL;
  };
  // The weights where this share begins and ends; false: there are fewer shares.  (A border is the same number in both of
  // its shares, and that is all that has to hold: 32-bit floats, which do not decrease with c.)
  auto borders = [&](long long total, long long& w0, long long& w1) {
    const int least = Row::unit(a);
    const int shares = total >= (long long)least * ctas ? ctas : max((int)total / least, 1);
    if (cta >= shares) return false;
    const float each = __fdividef(1.f, (float)shares), all = (float)total;
    w0 = (long long)(all * ((float)cta * each));
    w1 = cta + 1 == shares ? total : (long long)(all * ((float)(cta + 1) * each));
    return true;
  };
  long long* sums = reinterpret_cast<long long*>(scratch);  // a sum a warp
  Found* found = reinterpret_cast<Found*>(scratch + 256);
  Cut* cuts = reinterpret_cast<Cut*>(scratch + 384);
  // Up to 32 sequences are one warp's work, the others wait; up to kThreads are weighed and added up once.  (With all warps'
  // barriers and two scans this took 3.8 to 5.5 us from a kernel's start, now 2.7 to 3.4: mostly code read for the first
  // time.  One token over 700 keys 22.1 -> 20.7 us.)
  const bool few = s.B <= 32;
  Seq q{};  // of sequence threadIdx.x, if there are no more than threads
  if (!few || warp == 0) {
    if (threadIdx.x < 2) {
      found[threadIdx.x].b = -1;
      cuts[threadIdx.x] = Cut{s.B, 0, 0, 0};
    }
    __syncwarp();
    auto scan = [&](long long x, long long& all) {  // sum of the threads before this one; `all`: of all
      long long run = x;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      if (few) {
        all = __shfl_sync(0xffffffffu, run, 31);
        return run - x;
      }
      __syncthreads();
      if (lane == 31) sums[warp] = run;
      __syncthreads();
      long long ahead = 0;
      all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) ahead += sums[w];
        all += sums[w];
      }
      return ahead + run - x;
    };
    long long w = 0, at = 0, total = 0, all, w0 = 0, w1 = 0;
    auto mark = [&](int b) {  // the sequences that the share begins and ends in
      if (w > 0 && w0 >= at && w0 < at + w) found[0] = Found{q, w0 - at, b};
      if (w > 0 && w1 >= at && w1 < at + w) found[1] = Found{q, w1 - at, b};
    };
#pragma unroll 1
    for (int b0 = 0; b0 < s.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      w = b < s.B ? weigh(b, q, true) : 0;
      at = total + scan(w, all);
      total += all;
    }
    if (borders(total, w0, w1)) {
      if (s.B <= kThreads) {
        mark(threadIdx.x);
      } else {
        long long done = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < s.B; b0 += kThreads) {
          const int b = b0 + threadIdx.x;
          w = b < s.B ? weigh(b, q, false) : 0;
          at = done + scan(w, all);
          mark(b);
          done += all;
        }
      }
    }
    if (few) __syncwarp();
    else __syncthreads();
    if (threadIdx.x < 2 && found[threadIdx.x].b >= 0) {
      const Found f = found[threadIdx.x];
      cuts[threadIdx.x] = cut_at<Row>(a, f.q, f.w, f.b);
    }
  }
  __syncthreads();
  Share r{cuts[0], cuts[1], nullptr};
  const int held = min(r.to.b, s.B - 1) - r.from.b + 1;  // its sequences (none: from.b = B)
  Seq* kept = held <= kKept ? reinterpret_cast<Seq*>(kept_smem) : spill + r.from.b + cta;
  for (int b = r.from.b + threadIdx.x; b < r.from.b + held && s.B > kThreads; b += kThreads)
    kept[b - r.from.b] = load_seq<kPaged>(s, b);
  if (s.B <= kThreads && (int)threadIdx.x >= r.from.b && (int)threadIdx.x < r.from.b + held)
    kept[threadIdx.x - r.from.b] = q;
  r.kept = kept;
  return r;  // the caller's barrier makes `kept` visible
}

// Walks the items of a share.
template <class Row>
struct Walk {
  Cut at, end;
  const Seq* kept;
  int base, j0, j1, np;  // inner tiles j0 .. j1 - 1 of this part
  Seq q;
  bool part, first;  // part: of an item that was cut
  __device__ __forceinline__ explicit Walk(const Share& s)
      : at(s.from), end(s.to), kept(s.kept), base(s.from.b), j0(s.from.j), j1(0), np(-1), part(false), first(true) {
    at.j = 0;
  }
  __device__ __forceinline__ bool next(const SeqArgs& a) {
    if (!first) {
      ++at.p;
      j0 = 0;
    }
    first = false;
    while (true) {
      if (at.b >= a.s.B || at.b > end.b) return false;
      if (np < 0) {
        q = kept[at.b - base];
        np = Row::tiles(a, q);
      }
      if (at.p >= np) {
        at.p = 0;
        ++at.h;
      }
      if (np > 0 && at.h < a.s.Hk) break;
      at.h = at.p = 0;
      ++at.b;
      np = -1;
    }
    const bool last = same_item(at, end);
    if (!before(at, end) && !(last && end.j > 0)) return false;
    const int nt = Row::inner(a, q, at.p);
    j1 = last ? end.j : nt;
    part = j0 > 0 || j1 < nt;
    return true;
  }
};

// The parts of an item that was cut, for the kernel that joins them: block c - 1 takes the item that CTA c's share begins
// inside of, if no earlier share does.  Part 2 k + 1 is the tail of CTA k's share, 2 k its head; f(part) in order.
__device__ __forceinline__ bool leads(const Cut* first, int c, int B) {
  return first[c].b < B && first[c].j > 0 && !(same_item(first[c], first[c - 1]) && first[c - 1].j > 0);
}
// (The whole warp calls; f gets kBatch parts at a time, so that their loads are in flight together, the last batch filled
// up with -1.)
constexpr int kBatch = 4;
template <typename F>
__device__ __forceinline__ void each_part(const Cut* first, int c, int ctas, int nt, F&& f) {
  const int lane = threadIdx.x & 31;
  const Cut me = first[c];
  int ids[kBatch] = {2 * (c - 1) + 1, -1, -1, -1}, n = 1;
  for (int k0 = c;; k0 += 32) {
    const int k = k0 + lane;
    bool same = false, some = false;
    if (k < ctas) {
      const Cut x = first[k], y = first[min(k + 1, ctas - 1)];
      same = same_item(x, me);
      some = same && (k + 1 < ctas && same_item(y, me) ? y.j : nt) > x.j;
    }
    const uint32_t all = __ballot_sync(0xffffffffu, same);
    for (uint32_t left = __ballot_sync(0xffffffffu, some); left; left &= left - 1) {
      if (n == kBatch) {
        f(ids);
        n = 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) ids[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (u == n) ids[u] = 2 * (k0 + __ffs(left) - 1);
      ++n;
    }
    if (all != 0xffffffffu) break;
  }
  f(ids);
}
__device__ __forceinline__ int part_of(int cta, int j0) { return 2 * cta + (j0 > 0 ? 0 : 1); }

// ---------------------------------------------------------------------------
// Host: the checks that the calls share.
int check_seqs(const char* fn, const uaa_seqs* s, bool paged, bool bwd = false) {
  if (!s) return set_error(UAA_ERR_INVALID_ARG, "%s: the arguments are NULL", fn);
  if (s->B < 0 || s->T < 0 || s->Tk < 0 || s->Hq < 0 || s->Hk < 0)
    return set_error(UAA_ERR_INVALID_ARG, "%s: negative size B=%d T=%d Tk=%d Hq=%d Hk=%d", fn, s->B, s->T, s->Tk, s->Hq,
                     s->Hk);
  if (s->D != 64 && s->D != 128)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: D=%d (only 64 and 128 are built)", fn, s->D);
  if (s->dtype != UAA_BF16 && s->dtype != UAA_FP16)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: dtype %d (bf16 and fp16 are built)", fn, s->dtype);
  if (s->Hk == 0 || s->Hq == 0 || s->Hq % s->Hk)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d query heads over %d key heads", fn, s->Hq, s->Hk);
  if (s->Hq / s->Hk > 128)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: %d query heads a key head (128 at most)", fn, s->Hq / s->Hk);
  if (s->B > 65535 || s->Hq > 65535) return set_error(UAA_ERR_UNSUPPORTED, "%s: B and Hq must be <= 65535", fn);
  if ((long long)s->T * s->Hq >= (1LL << 32) - 1 || (long long)s->Tk * s->Hk >= (1LL << 32) - 1)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: 2^32 rows of one head or more", fn);
  if (s->T > kMostTokens || s->Tk > kMostTokens || (paged && (long long)s->width * s->page > kMostTokens))
    return set_error(UAA_ERR_UNSUPPORTED, "%s: more than 2^30 tokens", fn);
  if (!(s->scale > 0.f) || !isfinite(s->scale))
    return set_error(UAA_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
  if ((s->B == 0 && !s->rest) || (s->T == 0 && !(bwd && s->Tk > 0))) return UAA_OK;
  int st;
  const bool keys = paged ? s->pages > 0 : s->Tk > 0;
  if (keys && ((st = check_dev_ptr(fn, "k", s->k)) || (st = check_dev_ptr(fn, "v", s->v)))) return st;
  if (s->T > 0) {
    if ((st = check_dev_ptr(fn, "q", s->q)) || (st = check_dev_ptr(fn, "out", s->out))) return st;
    if (!s->lse || (reinterpret_cast<uintptr_t>(s->lse) & 3u))
      return set_error(UAA_ERR_INVALID_ARG, "%s: lse is NULL or not 4-byte aligned", fn);
  }
  if (!s->starts || ((reinterpret_cast<uintptr_t>(s->starts) | reinterpret_cast<uintptr_t>(s->starts_k)) & 3u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: starts is NULL or not 4-byte aligned", fn);
  // what a tensor map takes: strides of whole 16-byte pieces below 2^40 bytes
  auto stride = [&](const char* name, long long x) {
    if (x <= 0 || x % 8 || x >= (1LL << 39))
      return set_error(UAA_ERR_INVALID_ARG, "%s: a stride of %s is %lld elements (positive multiples of 8)", fn, name, x);
    return (int)UAA_OK;
  };
  if ((st = stride("q", s->q_row)) || (st = stride("q", s->q_head)) || (st = stride("k", s->k_row)) ||
      (st = stride("k", s->k_head)) || (st = stride("v", s->v_row)) || (st = stride("v", s->v_head)))
    return st;
  if (paged) {
    if (s->pages < 0 || s->width < 0 || s->table_rows < 0)
      return set_error(UAA_ERR_INVALID_ARG, "%s: negative size pages=%d width=%d table_rows=%d", fn, s->pages, s->width,
                       s->table_rows);
    if (s->page != 16 && s->page != 32 && s->page != 64 && (s->page < 128 || s->page % 128 || s->page > 65536))
      return set_error(UAA_ERR_UNSUPPORTED, "%s: pages of %d tokens (16, 32, 64 or a multiple of 128)", fn, s->page);
    if ((st = stride("k", s->k_page)) || (st = stride("v", s->v_page))) return st;
    if (!s->table || !s->lens || ((reinterpret_cast<uintptr_t>(s->table) | reinterpret_cast<uintptr_t>(s->lens) |
                                   reinterpret_cast<uintptr_t>(s->seqs)) & 3u))
      return set_error(UAA_ERR_INVALID_ARG, "%s: table or lens is NULL, or table, lens or seqs not 4-byte aligned", fn);
    if (!s->seqs && s->B > s->table_rows)
      return set_error(UAA_ERR_INVALID_ARG, "%s: %d sequences over a table of %d rows", fn, s->B, s->table_rows);
  }
  return UAA_OK;
}

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess || n <= 0)
    return 148;
  return n;
}

SeqArgs seq_args(const uaa_seqs& s) {
  SeqArgs a{};
  a.s = s;
  a.g = s.Hq / s.Hk;
  a.TT = 128 / a.g;
  return a;
}

}  // namespace
}  // namespace uaa
