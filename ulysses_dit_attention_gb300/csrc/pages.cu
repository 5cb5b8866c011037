// The pages of a key and value cache: who holds which page is kept on the host
// (UAA_PAGES below); the device gets the changes of its table, copies of shared or
// moved pages, and the rows of new tokens.
//
// Table changes travel as kernel arguments, runs of equal or consecutive entries,
// and so do the moves of a copy: no staging buffer that must outlive the call, no
// copy from pageable memory, one launch each for up to kMany of them.
//
// Bound of the copies and of the row writes: memory, each byte read and written
// once; of a page only the rows that a sequence has filled are copied.  Measured on a
// GB300: 24 sequences that end, 24 others written to their places and the rest closed
// up, 921 MB in four layers of 8 heads of 128: 175 us, 5.3 TB/s.  Calls of a few pages
// are launches: a fork of 8 sequences by 5, with one token more for each, is 35 MB in
// 9 launches, 116 to 131 us, nearly all of it on the host.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <mutex>
#include <new>
#include <unordered_map>
#include <vector>

#include "uaa_common.cuh"

namespace uaa {

int check_dev_ptr(const char* fn, const char* name, const void* p);

namespace {

// ---------------------------------------------------------------------------
// Device side
struct Edit {  // entries at .. at + count - 1 of a target: value, value + step, ...
  int at;
  uint32_t meta;  // count << 3 | step << 2 | target
  int value;
};
enum { kTable = 0, kLens = 1, kStarts = 2, kSeqs = 3 };
struct Move {  // the first `rows` rows of page src to page dst, in every layer
  int src, dst, rows;
};
// Entries of one launch: few in the usual 4 KB of arguments, many in 32 KB.
constexpr int kFew = 256, kMany = 2600;

template <int N>
struct EditArgs {
  int32_t* to[4];
  int n;
  Edit e[N];
};
template <int N>
struct MoveArgs {
  uint4 *k, *v;
  long long layer, page;  // strides in 16-byte pieces
  int row, n;             // pieces of a row
  Move m[N];
};
static_assert(sizeof(EditArgs<kMany>) <= 32764 && sizeof(MoveArgs<kMany>) <= 32764, "kernel arguments");

template <int N>
__global__ void __launch_bounds__(256) table_edit_kernel(const __grid_constant__ EditArgs<N> a) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= a.n) return;
  const Edit e = a.e[i];
  int32_t* to = a.to[e.meta & 3u] + e.at;
  const int count = (int)(e.meta >> 3), step = (e.meta >> 2) & 1u;
  for (int x = threadIdx.x & 31; x < count; x += 32) to[x] = e.value + step * x;
}

// Block (move, part, layer and tensor): kCopy pieces a thread in flight.
constexpr int kCopy = 8, kCopyThreads = 256;
template <int N>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const __grid_constant__ MoveArgs<N> a) {
  const Move m = a.m[blockIdx.x];
  uint4* pool = (blockIdx.z & 1 ? a.v : a.k) + (blockIdx.z >> 1) * a.layer;
  const uint4* src = pool + m.src * a.page;
  uint4* dst = pool + m.dst * a.page;
  const long long pieces = (long long)m.rows * a.row;
  for (long long i = (long long)blockIdx.y * (kCopy * kCopyThreads) + threadIdx.x; i < pieces;
       i += (long long)gridDim.y * (kCopy * kCopyThreads)) {
    uint4 x[kCopy];
#pragma unroll
    for (int u = 0; u < kCopy; ++u)
      if (i + u * kCopyThreads < pieces) x[u] = __ldcs(src + i + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kCopy; ++u)
      if (i + u * kCopyThreads < pieces) __stcs(dst + i + u * kCopyThreads, x[u]);
  }
}

// A warp takes a token: its page and row, then the keys and the values, 16 bytes a lane.
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ uaa_cache_rows a, DevCtx ctx) {
  const int lane = threadIdx.x & 31;
  const int pieces = a.D / 8, all = a.Hk * pieces;
  for (int t = blockIdx.x * 8 + (threadIdx.x >> 5); t < a.T; t += gridDim.x * 8) {
    // the last b with starts[b] <= t
    int lo = 0, hi = a.B;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.starts[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    if (lo >= a.B || a.starts[lo] > t) continue;  // behind the last sequence
    const int r = a.seqs ? a.seqs[lo] : lo;
    long long at = -1;
    int page = -1;
    if (r >= 0 && r < a.table_rows) {
      at = (long long)a.lens[r] - (min(a.starts[lo + 1], a.T) - t);
      if (at >= 0 && at < (long long)a.width * a.page) page = a.table[(size_t)r * a.width + at / a.page];
    }
    if (page < 0 || page >= a.pages) {
      if (lane == 0) atomicOr(ctx.status, kStatusBadPage);
      continue;
    }
    const int row = (int)(at % a.page);
    const char* k = static_cast<const char*>(a.k) + (size_t)t * a.k_row * 2;
    const char* v = static_cast<const char*>(a.v) + (size_t)t * a.v_row * 2;
    char* kp = static_cast<char*>(a.k_pages) + ((size_t)page * a.kp_page + (size_t)row * a.kp_row) * 2;
    char* vp = static_cast<char*>(a.v_pages) + ((size_t)page * a.vp_page + (size_t)row * a.vp_row) * 2;
    // kRows pieces of the keys and of the values in flight a lane
    constexpr int kRows = 4;
    for (int i0 = lane; i0 < all; i0 += 32 * kRows) {
      uint4 x[kRows], y[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int i = i0 + 32 * u, h = i / pieces, c = (i - h * pieces) * 16;
        if (i < all) {
          x[u] = __ldcs(reinterpret_cast<const uint4*>(k + (size_t)h * a.k_head * 2 + c));
          y[u] = __ldcs(reinterpret_cast<const uint4*>(v + (size_t)h * a.v_head * 2 + c));
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int i = i0 + 32 * u, h = i / pieces, c = (i - h * pieces) * 16;
        if (i < all) {
          *reinterpret_cast<uint4*>(kp + (size_t)h * a.kp_head * 2 + c) = x[u];
          *reinterpret_cast<uint4*>(vp + (size_t)h * a.vp_head * 2 + c) = y[u];
        }
      }
    }
  }
}

int check_pools(const char* fn, const uaa_pools* d, cudaStream_t stream) {
  if (!d) return UAA_OK;
  int st;
  if ((st = check_dev_ptr(fn, "k", d->k)) || (st = check_dev_ptr(fn, "v", d->v))) return st;
  if (!d->table || !d->lens || ((reinterpret_cast<uintptr_t>(d->table) | reinterpret_cast<uintptr_t>(d->lens)) & 3u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: table or lens is NULL or not 4-byte aligned", fn);
  if (d->layers < 1 || d->layers > 32767 || d->row_bytes < 16 || d->row_bytes % 16)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d layers of rows of %d bytes (a multiple of 16)", fn, d->layers,
                     d->row_bytes);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(stream, &capture);
  if (e != cudaSuccess) {
    cudaGetLastError();  // reported here, not by a later call's launch
    return set_error(UAA_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  }
  if (capture != cudaStreamCaptureStatusNone)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: not inside a graph capture: the pages are kept on the host", fn);
  return UAA_OK;
}

}  // namespace
}  // namespace uaa

using namespace uaa;

// ---------------------------------------------------------------------------
// Host side
struct uaa_pages {
  std::mutex mu;
  int pages, page, seqs, width, unused, hint;  // hint: no page below is free
  std::vector<int> refs;                       // holders of each page
  std::vector<int> held;                       // (seqs, width)
  std::vector<int> size;                       // tokens of each sequence
  // of the call in progress, kept so that a call allocates nothing once it has begun to change the rest
  std::vector<Edit> edits;
  std::vector<Move> moves;
  std::vector<unsigned> seen;  // the call that last named a sequence
  unsigned call = 0;
  bool lost = false;  // a launch failed when the host's side had changed: the device's side is another one

  int need(int tokens) const { return (int)(((long long)tokens + page - 1) / page); }
  int take() {
    while (refs[hint]) ++hint;
    refs[hint] = 1;
    --unused;
    return hint++;
  }
  void drop(int p) {
    if (--refs[p]) return;
    ++unused;
    hint = std::min(hint, p);
  }
  // Runs of the table's entries [from, to) of a row, and the row's length.
  void tell(int seq, int from, int to) {
    const int* row = held.data() + (size_t)seq * width;
    for (int i = from; i < to;) {
      int n = 1, step = 0;
      if (i + 1 < to && (row[i + 1] == row[i] || row[i + 1] == row[i] + 1)) {
        step = row[i + 1] - row[i];
        // -1, 0, 1, ... is not one run: -1 stands for no page
        if (row[i] < 0) step = 0;
        while (i + n < to && row[i + n] == row[i] + step * n) ++n;
      }
      edits.push_back({seq * width + i, (uint32_t)n << 3 | (uint32_t)step << 2 | kTable, row[i]});
      i += n;
    }
    edits.push_back({seq, 1u << 3 | kLens, size[seq]});
  }
  bool named(int seq) { return seen[seq] == call || (seen[seq] = call, false); }
  void begin() {
    edits.clear();
    moves.clear();
    if (++call == 0) {
      std::fill(seen.begin(), seen.end(), 0u);
      call = 1;
    }
  }
};

namespace {

std::atomic<int> g_fail_launch{-1};  // diagnostic: the launch of every call that is not made and counts as failed

// One launch of a call, its `index`-th.  What it returns is asked, not the last error: that may be an older call's.
template <typename A>
int send_one(const char* fn, void (*kernel)(A), dim3 grid, int threads, const A& a, int index, cudaStream_t s) {
  if (index == g_fail_launch.load(std::memory_order_relaxed))
    return set_error(UAA_ERR_CUDA, "%s: launch failed: left out by uaa_debug_fail_launch", fn);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e == cudaSuccess) return UAA_OK;
  cudaGetLastError();
  return set_error(UAA_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

template <int N>
int send_moves(const char* fn, const uaa_pools& d, const uaa_pages& p, const Move* m, int n, int index, cudaStream_t s) {
  MoveArgs<N> a;
  a.k = static_cast<uint4*>(d.k);
  a.v = static_cast<uint4*>(d.v);
  a.row = d.row_bytes / 16;
  a.page = (long long)a.row * p.page;
  a.layer = a.page * p.pages;
  a.n = n;
  std::copy(m, m + n, a.m);
  const long long parts = (a.page + kCopy * kCopyThreads - 1) / (kCopy * kCopyThreads);
  return send_one(fn, page_copy_kernel<N>, dim3(n, (unsigned)std::min(parts, 64LL), 2 * d.layers), kCopyThreads, a, index, s);
}

template <int N>
int send_edits(const char* fn, const uaa_pools& d, int32_t* starts, int32_t* seqs, const Edit* e, int n, int index,
               cudaStream_t s) {
  EditArgs<N> a;
  a.to[kTable] = d.table;
  a.to[kLens] = d.lens;
  a.to[kStarts] = starts;
  a.to[kSeqs] = seqs;
  a.n = n;
  std::copy(e, e + n, a.e);
  return send_one(fn, table_edit_kernel<N>, dim3((n + 7) / 8), 256, a, index, s);
}

// The call's copies and table changes, enqueued.  The host's side has changed already: a launch that fails leaves the two
// apart, and as the copies of shared pages may be among what is missing, the object takes no further call.
int send(const char* fn, uaa_pages& p, const uaa_pools* d, int32_t* starts, int32_t* seqs, cudaStream_t s) {
  if (!d) return UAA_OK;
  int index = 0;
  for (size_t i = 0; i < p.moves.size(); i += kMany, ++index) {
    const int n = (int)std::min(p.moves.size() - i, (size_t)kMany);
    const Move* m = p.moves.data() + i;
    const int st = n <= kFew ? send_moves<kFew>(fn, *d, p, m, n, index, s) : send_moves<kMany>(fn, *d, p, m, n, index, s);
    if (st) return p.lost = true, st;
  }
  for (size_t i = 0; i < p.edits.size(); i += kMany, ++index) {
    const int n = (int)std::min(p.edits.size() - i, (size_t)kMany);
    const Edit* e = p.edits.data() + i;
    const int st = n <= kFew ? send_edits<kFew>(fn, *d, starts, seqs, e, n, index, s)
                             : send_edits<kMany>(fn, *d, starts, seqs, e, n, index, s);
    if (st) return p.lost = true, st;
  }
  return UAA_OK;
}

int check_lost(const char* fn, const uaa_pages& p, const uaa_pools* d) {
  if (d && p.lost)
    return set_error(UAA_ERR_CUDA, "%s: a launch of an earlier call failed: the device's table is not the host's; "
                     "destroy the cache", fn);
  return UAA_OK;
}

int check_seq(const char* fn, const uaa_pages& p, int seq) {
  if (seq < 0 || seq >= p.seqs)
    return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d of %d", fn, seq, p.seqs);
  return UAA_OK;
}

int check_list(const char* fn, const uaa_pages* p, int n, const int* a, const int* b) {
  if (!p) return set_error(UAA_ERR_INVALID_ARG, "%s: the cache is NULL", fn);
  if (n < 0 || n > p->seqs) return set_error(UAA_ERR_INVALID_ARG, "%s: %d sequences of %d", fn, n, p->seqs);
  if (n > 0 && (!a || !b)) return set_error(UAA_ERR_INVALID_ARG, "%s: NULL array", fn);
  return UAA_OK;
}

// No C++ exception leaves the library.
template <typename F>
int guarded(const char* fn, F&& f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return set_error(UAA_ERR_INVALID_ARG, "%s: out of host memory", fn);
  } catch (...) {
    return set_error(UAA_ERR_INVALID_ARG, "%s: failed on the host", fn);
  }
}

}  // namespace

extern "C" int uaa_pages_create(uaa_pages** out, int pages, int page, int seqs, int width) {
  const char* fn = "uaa_pages_create";
  return guarded(fn, [&] {
    if (!out) return set_error(UAA_ERR_INVALID_ARG, "%s: out is NULL", fn);
    if (pages < 1 || seqs < 1 || width < 1)
      return set_error(UAA_ERR_INVALID_ARG, "%s: pages=%d seqs=%d width=%d must be positive", fn, pages, seqs, width);
    if (page != 16 && page != 32 && page != 64 && (page < 128 || page % 128 || page > 65536))
      return set_error(UAA_ERR_UNSUPPORTED, "%s: pages of %d tokens (16, 32, 64 or a multiple of 128)", fn, page);
    if ((long long)seqs * width > (1 << 28) || (long long)width * page > (1 << 30))
      return set_error(UAA_ERR_UNSUPPORTED, "%s: a table of %d x %d pages of %d tokens", fn, seqs, width, page);
    uaa_pages* p = new uaa_pages;
    try {
      p->pages = p->unused = pages;
      p->page = page;
      p->seqs = seqs;
      p->width = width;
      p->hint = 0;
      p->refs.assign(pages, 0);
      p->held.assign((size_t)seqs * width, -1);
      p->size.assign(seqs, 0);
      p->seen.assign(seqs, 0u);
    } catch (...) {
      delete p;
      throw;
    }
    *out = p;
    return (int)UAA_OK;
  });
}

extern "C" void uaa_pages_destroy(uaa_pages* p) { delete p; }

extern "C" int uaa_pages_append(uaa_pages* p, const uaa_pools* pools, int n, const int* seqs, const int* counts,
                                int32_t* starts, int32_t* seqs_dev, uaa_stream_t stream) {
  const char* fn = "uaa_pages_append";
  return guarded(fn, [&] {
    int st = check_list(fn, p, n, seqs, counts);
    if (!st && ((reinterpret_cast<uintptr_t>(starts) | reinterpret_cast<uintptr_t>(seqs_dev)) & 3u))
      st = set_error(UAA_ERR_INVALID_ARG, "%s: starts or seqs_dev is not 4-byte aligned", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (st || (st = check_pools(fn, pools, s))) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    if ((st = check_lost(fn, *p, pools))) return st;
    p->begin();
    long long want = 0, total = 0, entries = 0;
    std::unordered_map<int, int> left;  // holders of a shared last page, less those that this call takes off it
    for (int i = 0; i < n; ++i) {
      const int q = seqs[i];
      if ((st = check_seq(fn, *p, q))) return st;
      if (p->named(q)) return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d is named twice", fn, q);
      if (counts[i] < 0) return set_error(UAA_ERR_INVALID_ARG, "%s: %d tokens", fn, counts[i]);
      const long long len = (long long)p->size[q] + counts[i];
      if (len > (long long)p->width * p->page)
        return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d would have %lld tokens of %lld", fn, q, len,
                         (long long)p->width * p->page);
      total += counts[i];
      const int more = p->need((int)len) - p->need(p->size[q]);
      want += more;
      entries += more + 2;
      if (counts[i] && p->size[q] % p->page) {
        const int last = p->held[(size_t)q * p->width + p->size[q] / p->page];
        if (p->refs[last] > 1) {
          auto it = left.emplace(last, p->refs[last]).first;
          if (it->second > 1) {
            --it->second;
            ++want;
          }
        }
      }
    }
    if (total > INT_MAX) return set_error(UAA_ERR_UNSUPPORTED, "%s: %lld tokens at once", fn, total);
    if (want > p->unused)
      return set_error(UAA_ERR_NO_PAGES, "%s: %lld pages wanted, %d free", fn, want, p->unused);
    p->moves.reserve(n);
    p->edits.reserve((size_t)entries + 2 * (size_t)n + 2);
    long long at = 0;
    for (int i = 0; i < n; ++i) {
      const int q = seqs[i], old = p->size[q], filled = old % p->page;
      int* row = p->held.data() + (size_t)q * p->width;
      int from = p->need(old);
      if (counts[i] && filled && p->refs[row[from - 1]] > 1) {
        const int src = row[--from], dst = p->take();
        p->drop(src);
        row[from] = dst;
        p->moves.push_back({src, dst, filled});
      }
      const int first = filled && counts[i] && from < p->need(old) ? from + 1 : from;
      p->size[q] = old + counts[i];
      const int to = p->need(p->size[q]);
      for (int x = first; x < to; ++x) row[x] = p->take();
      p->tell(q, from, to);
    }
    if (pools && starts) {  // runs of one step: 0, 1, 2, ... where every count is 1, or single sums
      for (int i = 0; i <= n;) {
        int run = 1;
        long long x = at;
        while (i + run <= n && counts[i + run - 1] == 1) ++run, ++x;
        p->edits.push_back({i, (uint32_t)run << 3 | 1u << 2 | kStarts, (int)at});
        i += run;
        if (i <= n) at = x + counts[i - 1];
      }
    }
    if (pools && seqs_dev) {
      for (int i = 0; i < n;) {
        int run = 1;
        while (i + run < n && seqs[i + run] == seqs[i] + run) ++run;
        p->edits.push_back({i, (uint32_t)run << 3 | 1u << 2 | kSeqs, seqs[i]});
        i += run;
      }
    }
    return send(fn, *p, pools, starts, seqs_dev, s);
  });
}

extern "C" int uaa_pages_fork(uaa_pages* p, const uaa_pools* pools, int n, const int* parents, const int* children,
                              uaa_stream_t stream) {
  const char* fn = "uaa_pages_fork";
  return guarded(fn, [&] {
    int st = check_list(fn, p, n, parents, children);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (st || (st = check_pools(fn, pools, s))) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    if ((st = check_lost(fn, *p, pools))) return st;
    p->begin();
    size_t entries = 0;
    for (int i = 0; i < n; ++i) {
      const int c = children[i];
      if ((st = check_seq(fn, *p, parents[i])) || (st = check_seq(fn, *p, c))) return st;
      if (p->named(c)) return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d is named twice", fn, c);
      if (p->size[c]) return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d is not empty", fn, c);
      entries += p->need(p->size[parents[i]]) + 1;
    }
    for (int i = 0; i < n; ++i)
      if (p->seen[parents[i]] == p->call)
        return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d is both a parent and a child", fn, parents[i]);
    p->edits.reserve(entries);
    for (int i = 0; i < n; ++i) {
      const int* from = p->held.data() + (size_t)parents[i] * p->width;
      int* row = p->held.data() + (size_t)children[i] * p->width;
      const int pages = p->need(p->size[parents[i]]);
      for (int x = 0; x < pages; ++x) ++p->refs[row[x] = from[x]];
      p->size[children[i]] = p->size[parents[i]];
      p->tell(children[i], 0, pages);
    }
    return send(fn, *p, pools, nullptr, nullptr, s);
  });
}

extern "C" int uaa_pages_truncate(uaa_pages* p, const uaa_pools* pools, int n, const int* seqs, const int* lens,
                                  uaa_stream_t stream) {
  const char* fn = "uaa_pages_truncate";
  return guarded(fn, [&] {
    int st = check_list(fn, p, n, seqs, lens);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (st || (st = check_pools(fn, pools, s))) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    if ((st = check_lost(fn, *p, pools))) return st;
    p->begin();
    for (int i = 0; i < n; ++i) {
      const int q = seqs[i];
      if ((st = check_seq(fn, *p, q))) return st;
      if (p->named(q)) return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d is named twice", fn, q);
      if (lens[i] < 0 || lens[i] > p->size[q])
        return set_error(UAA_ERR_INVALID_ARG, "%s: sequence %d has %d tokens, not %d", fn, q, p->size[q], lens[i]);
    }
    p->edits.reserve(2 * (size_t)n);
    for (int i = 0; i < n; ++i) {
      const int q = seqs[i], from = p->need(lens[i]), to = p->need(p->size[q]);
      int* row = p->held.data() + (size_t)q * p->width;
      for (int x = from; x < to; ++x) {
        p->drop(row[x]);
        row[x] = -1;
      }
      if (p->size[q] == lens[i]) continue;
      p->size[q] = lens[i];
      p->tell(q, from, to);
    }
    return send(fn, *p, pools, nullptr, nullptr, s);
  });
}

extern "C" int uaa_pages_compact(uaa_pages* p, const uaa_pools* pools, uaa_stream_t stream) {
  const char* fn = "uaa_pages_compact";
  return guarded(fn, [&] {
    if (!p) return set_error(UAA_ERR_INVALID_ARG, "%s: the cache is NULL", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int st = check_pools(fn, pools, s);
    if (st) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    if ((st = check_lost(fn, *p, pools))) return st;
    p->begin();
    const int used = p->pages - p->unused;
    std::unordered_map<int, size_t> to;  // page -> its move
    int hole = 0;
    for (int x = used; x < p->pages; ++x) {
      if (!p->refs[x]) continue;
      while (p->refs[hole]) ++hole;
      to.emplace(x, p->moves.size());
      p->moves.push_back({x, hole++, 0});
    }
    if (p->moves.empty()) return (int)UAA_OK;
    size_t entries = 0;
    for (const Move& m : p->moves) entries += p->refs[m.src];
    p->edits.reserve(2 * entries);
    for (const Move& m : p->moves) std::swap(p->refs[m.src], p->refs[m.dst]);
    p->hint = used;
    for (int q = 0; q < p->seqs; ++q) {
      int* row = p->held.data() + (size_t)q * p->width;
      const int pages = p->need(p->size[q]);
      for (int x = 0; x < pages;) {
        int e = x;  // a run of moved pages
        for (; e < pages && row[e] >= used; ++e) {
          Move& m = p->moves[to.find(row[e])->second];
          m.rows = std::max(m.rows, std::min(p->page, p->size[q] - e * p->page));
          row[e] = m.dst;
        }
        if (e > x) p->tell(q, x, e);
        x = e + 1;
      }
    }
    return send(fn, *p, pools, nullptr, nullptr, s);
  });
}

extern "C" void uaa_debug_fail_launch(int n) { g_fail_launch.store(n < 0 ? -1 : n); }

extern "C" int uaa_pages_row(uaa_pages* p, int seq, int* out, int most) {
  const char* fn = "uaa_pages_row";
  if (!p) return set_error(UAA_ERR_INVALID_ARG, "%s: the cache is NULL", fn);
  return guarded(fn, [&] {
    if (int st = check_seq(fn, *p, seq)) return st;
    std::lock_guard<std::mutex> lock(p->mu);
    const int n = std::min(p->need(p->size[seq]), most);
    if (out && n > 0) std::copy_n(p->held.data() + (size_t)seq * p->width, n, out);
    return p->size[seq];
  });
}

extern "C" int uaa_pages_free(uaa_pages* p) {
  const char* fn = "uaa_pages_free";
  if (!p) return set_error(UAA_ERR_INVALID_ARG, "%s: the cache is NULL", fn);
  return guarded(fn, [&] {
    std::lock_guard<std::mutex> lock(p->mu);
    return p->unused;
  });
}

extern "C" int uaa_cache_write(const uaa_cache_rows* args, uaa_stream_t stream) {
  const char* fn = "uaa_cache_write";
  if (!args) return set_error(UAA_ERR_INVALID_ARG, "%s: the arguments are NULL", fn);
  const uaa_cache_rows& a = *args;
  if (a.B < 0 || a.T < 0 || a.Hk < 0 || a.pages < 0 || a.width < 0 || a.table_rows < 0)
    return set_error(UAA_ERR_INVALID_ARG, "%s: negative size B=%d T=%d Hk=%d pages=%d width=%d", fn, a.B, a.T, a.Hk,
                     a.pages, a.width);
  if (a.D < 8 || a.D % 8) return set_error(UAA_ERR_UNSUPPORTED, "%s: D=%d (a multiple of 8)", fn, a.D);
  if (a.page < 1) return set_error(UAA_ERR_INVALID_ARG, "%s: pages of %d tokens", fn, a.page);
  if (a.B == 0 || a.T == 0 || a.Hk == 0) return UAA_OK;
  int st;
  if ((st = check_dev_ptr(fn, "k", a.k)) || (st = check_dev_ptr(fn, "v", a.v)) ||
      (st = check_dev_ptr(fn, "k_pages", a.k_pages)) || (st = check_dev_ptr(fn, "v_pages", a.v_pages)))
    return st;
  if (!a.starts || !a.table || !a.lens ||
      ((reinterpret_cast<uintptr_t>(a.starts) | reinterpret_cast<uintptr_t>(a.seqs) |
        reinterpret_cast<uintptr_t>(a.table) | reinterpret_cast<uintptr_t>(a.lens)) & 3u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: starts, table or lens is NULL, or one of them or seqs not 4-byte aligned", fn);
  if (!a.seqs && a.B > a.table_rows)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d sequences over a table of %d rows", fn, a.B, a.table_rows);
  for (long long x : {a.k_row, a.k_head, a.v_row, a.v_head, a.kp_page, a.kp_row, a.kp_head, a.vp_page, a.vp_row, a.vp_head})
    if (x < 0 || x % 8) return set_error(UAA_ERR_INVALID_ARG, "%s: a stride is %lld elements (multiples of 8)", fn, x);
  DevCtx ctx;
  if ((st = get_dev_ctx(&ctx))) return st;
  const int blocks = (int)std::min(((long long)a.T + 7) / 8, 152LL * 64);
  cache_write_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(a, ctx);
  return check_launch(fn);
}
