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

struct SeqArgs {
  uaa_seqs s;
  int g;   // query heads of a key head
  int TT;  // tokens of a tile of 128 rows, a row being one head of one token
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
__device__ __forceinline__ int keys_of(const uaa_seqs& s, const Seq& q, int i) {
  return s.causal ? held_in(q.m - q.n + i + 1, 0, q.m) : q.m;
}

// The sequence that token t belongs to, or -1 behind the last one (binary search; starts must not decrease).
__device__ __forceinline__ int seq_of_token(const int* starts, int B, int t) {
  int lo = 0, hi = B;  // the last b with starts[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo < B && starts[lo] <= t ? lo : -1;
}

__device__ __forceinline__ float load16(const void* p, size_t at, int fp16) {
  return fp16 ? __half2float(static_cast<const __half*>(p)[at]) : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void store16(void* p, size_t at, float x, int fp16) {
  if (fp16) static_cast<__half*>(p)[at] = __float2half_rn(x);
  else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(x);
}

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
  if (!(s->scale > 0.f) || !isfinite(s->scale))
    return set_error(UAA_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
  if (s->B == 0 || (s->T == 0 && !(bwd && s->Tk > 0))) return UAA_OK;
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
