// Rotary positions: pairs of columns of every head are turned by an angle that
// grows with the token's position, Q and K in one launch, and the transpose of
// that map for the gradients.
//
// Pair i of a head (columns i and i + R/2, or 2i and 2i + 1) turns by
//   a = 2 pi * frac(position[axis_i] * turns_i),
//   y0 = m (x0 cos a - x1 sin a),  y1 = m (x0 sin a + x1 cos a),
// and columns R..D-1 are copied.  The transpose has -sin a.
//
// turns_i (turns per position) is kept as a 64-bit fixed-point fraction of a
// turn, so the 64-bit product with the position drops whole turns by itself and
// costs one integer multiplication, where a 32-bit angle of a position near 2^18
// would be off by 2^-6 radians and a 64-bit floating-point one would use the FP64
// pipe, 1/64 of the FP32 rate here.  turns_i itself is computed in 64-bit floating
// point, at most 2^-2.6 turns with 53 bits: its error, up to 2^-55 turns (against
// 200 bits; widths 2 to 256, bases 100 to 10^6, all scalings), is multiplied by the
// position, 2^-24 turns at 2^31.  The upper 32 bits of the product, as a signed
// number of half turns and rounded to 24 bits (2^-26 turns), go to sincospif.
//
// Bound: HBM.  Every element is read once and written once; the angles are
// computed once per token by the block (R/2 of them, in shared memory) and used
// by all heads of Q and K.  Q and K of 27280 x 40 x 128 in bf16: 184 us a pass
// interleaved, 170 in halves, 6.1 and 6.6 TB/s, 0.91 and 0.98 of a copy's rate.
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>

#include "uaa_common.cuh"

namespace uaa {
namespace {

constexpr int kThreads = 128;  // fewer threads wait for a token's angles at a time (256: 189 us instead of those 170)
constexpr int kMaxPairs = UAA_ROTARY_MAX_PAIRS;
constexpr int kMaxTokens = 16;       // tokens of one block (shared memory: kMaxTokens * kMaxPairs * 8 bytes at most)
constexpr int kMaxSmemPairs = 2048;  // pairs whose cosine and sine a block holds: 16 KB

struct RotTensor {
  const void* x;
  void* y;
  long long xb, xs, xh, yb, ys, yh;  // batch, token and head strides in elements; columns are contiguous
  int H;
  long long extent;  // elements from the first of y to its last
};

struct RotArgs {
  RotTensor t[2];
  const void* positions;  // NULL: position = start + s, the same on every axis
  long long start, pb, ps;
  int pos64;              // positions are 64-bit
  int B, S, D, inverse;
  uint32_t tokens, tokens_per_block, units, pair_units;  // units of a head row; the first pair_units hold pairs
  uaa_rotary_plan plan;
  DevCtx ctx;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements, moved as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
  T e[V];
};

// One pair, with the same roundings in every kernel; c = (cos a, sin a) * m
template <typename T>
__device__ __forceinline__ void turn_pair(float2 c, T& u, T& w) {
  const float x0 = to_f32<T>(u), x1 = to_f32<T>(w);
  u = from_f32<T>(fmaf(x0, c.x, -(x1 * c.y)));
  w = from_f32<T>(fmaf(x0, c.y, x1 * c.x));
}

// (cos a, sin a) * m of every pair of nt tokens
__device__ __forceinline__ void angles(const RotArgs& a, uint32_t t0, uint32_t nt, float2* cs) {
  const int pairs = a.plan.rot / 2;
  for (uint32_t i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const uint32_t tok = t0 + i / pairs, p = i % pairs;
    const uint32_t b = tok / a.S, s = tok - b * a.S;
    long long pos = a.start + s;
    if (a.positions) {
      const long long at = b * a.pb + s * a.ps + a.plan.axis[p];
      pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
    }
    const uint64_t turn = static_cast<uint64_t>(pos) * a.plan.turns[p];
    // the fraction of a turn in (-1/2, 1/2], in half turns: 32 bits, rounded to 24 by the conversion
    const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
    float sn, cn;
    sincospif(half_turns, &sn, &cn);
    cs[i] = make_float2(cn * a.plan.magnitude, (a.inverse ? -sn : sn) * a.plan.magnitude);
  }
}

// Row h of token tok: the tensor that holds it, its input and its output
template <typename T>
__device__ __forceinline__ const RotTensor& locate(const RotArgs& a, uint32_t tok, uint32_t h, const T** x, T** y) {
  const uint32_t b = tok / a.S, s = tok - b * a.S;
  const bool second = h >= static_cast<uint32_t>(a.t[0].H);
  const RotTensor& t = a.t[second ? 1 : 0];
  if (second) h -= a.t[0].H;
  *x = static_cast<const T*>(t.x) + (b * t.xb + s * t.xs + h * t.xh);
  *y = static_cast<T*>(t.y) + (b * t.yb + s * t.ys + h * t.yh);
  return t;
}

// A store of a vector, range-checked in debug builds.
template <typename T, int V>
__device__ __forceinline__ void store(const RotArgs& a, const RotTensor& t, T* at, const Vec<T, V>& v) {
  if (guard_store(a.ctx, at - static_cast<T*>(t.y), V, t.extent)) *reinterpret_cast<Vec<T, V>*>(at) = v;
}

// One thread takes units: of V pairs in two runs of V columns (halves, or V = 1), of V / 2 interleaved pairs in one run,
// or of V copied columns.
template <typename T, int V, bool kHalf>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
  extern __shared__ float2 cs[];  // (cos a, sin a) * m of this block's tokens
  const int pairs = a.plan.rot / 2;
  const uint32_t heads = a.t[0].H + a.t[1].H;
  for (uint32_t t0 = blockIdx.x * a.tokens_per_block; t0 < a.tokens; t0 += gridDim.x * a.tokens_per_block) {
    const uint32_t nt = a.tokens - t0 < a.tokens_per_block ? a.tokens - t0 : a.tokens_per_block;
    angles(a, t0, nt, cs);
    __syncthreads();
    const uint32_t work = nt * heads * a.units;
    for (uint32_t i = threadIdx.x; i < work; i += kThreads) {
      const uint32_t row = i / a.units, u = i - row * a.units;
      const uint32_t lt = row / heads;
      const T* x;
      T* y;
      const RotTensor& t = locate(a, t0 + lt, row - lt * heads, &x, &y);
      using VT = Vec<T, V>;
      if (u < a.pair_units) {
        if constexpr (kHalf || V == 1) {
          const int c0 = kHalf ? u * V : 2 * u, c1 = kHalf ? c0 + pairs : c0 + 1;
          VT v0 = *reinterpret_cast<const VT*>(x + c0), v1 = *reinterpret_cast<const VT*>(x + c1);
          const float2* w = cs + lt * pairs + u * V;
#pragma unroll
          for (int e = 0; e < V; ++e) turn_pair(w[e], v0.e[e], v1.e[e]);
          store(a, t, y + c0, v0);
          store(a, t, y + c1, v1);
        } else {
          VT v = *reinterpret_cast<const VT*>(x + u * V);
          const float2* w = cs + lt * pairs + u * (V / 2);
#pragma unroll
          for (int e = 0; e < V / 2; ++e) turn_pair(w[e], v.e[2 * e], v.e[2 * e + 1]);
          store(a, t, y + u * V, v);
        }
      } else {
        const int c = a.plan.rot + (u - a.pair_units) * V;
        store(a, t, y + c, *reinterpret_cast<const VT*>(x + c));
      }
    }
    __syncthreads();  // the next tokens' angles replace these
  }
}

// Rows of whole 16-byte vectors whose pairs are not: rot / 2 or D - rot is not a multiple of the vector's elements.  A
// warp takes as many rows as its lanes hold, one vector a lane.  Interleaved pairs lie in one lane; halves are read from
// and written to the rows in shared memory, pair by pair, so a row may be turned in place.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kThreads) rotary_rows_kernel(const __grid_constant__ RotArgs a) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ float2 cs[];
  __shared__ Vec<T, E> stage[kHalf ? kThreads : 1];
  const uint32_t pairs = a.plan.rot / 2, heads = a.t[0].H + a.t[1].H;
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t L = a.units, rw = 32 / L, r = lane / L, j = lane % L;  // vectors of a row, rows of a warp
  Vec<T, E>* mine = stage + warp * 32;
  for (uint32_t t0 = blockIdx.x * a.tokens_per_block; t0 < a.tokens; t0 += gridDim.x * a.tokens_per_block) {
    const uint32_t nt = a.tokens - t0 < a.tokens_per_block ? a.tokens - t0 : a.tokens_per_block;
    angles(a, t0, nt, cs);
    __syncthreads();
    const uint32_t rows = nt * heads;
    for (uint32_t r0 = warp * rw; r0 < rows; r0 += kThreads / 32 * rw) {
      const uint32_t row = r0 + r, lt = row / heads;
      const bool active = r < rw && row < rows;
      const T* x;
      T* y = nullptr;
      Vec<T, E> v;
      const RotTensor* t = nullptr;
      if (active) {
        t = &locate(a, t0 + lt, row - lt * heads, &x, &y);
        v = *reinterpret_cast<const Vec<T, E>*>(x + j * E);
      }
      if constexpr (kHalf) {
        if (active) mine[lane] = v;
        __syncwarp();
        for (uint32_t n = 0; n < rw && r0 + n < rows; ++n) {
          T* buf = mine[n * L].e;
          const float2* w = cs + (r0 + n) / heads * pairs;
          for (uint32_t p = lane; p < pairs; p += 32) {
            T u = buf[p], o = buf[p + pairs];
            turn_pair(w[p], u, o);
            buf[p] = u;
            buf[p + pairs] = o;
          }
        }
        __syncwarp();
        if (active) v = mine[lane];
      } else if (active) {
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const uint32_t p = j * (E / 2) + e;
          if (p >= pairs) continue;
          turn_pair(cs[lt * pairs + p], v.e[2 * e], v.e[2 * e + 1]);
        }
      }
      if (active) store(a, *t, y + j * E, v);
    }
    __syncthreads();  // the next tokens' angles replace these
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess || n <= 0)
    return 148;
  return n;
}

template <typename T, int V>
int launch_v(const RotArgs& a, int grid, size_t smem, cudaStream_t s) {
  if (a.plan.layout == UAA_ROTARY_HALF)
    rotary_kernel<T, V, true><<<grid, kThreads, smem, s>>>(a);
  else
    rotary_kernel<T, V, false><<<grid, kThreads, smem, s>>>(a);
  return check_launch("uaa_rotary");
}

// Do all rows begin at multiples of v elements?
bool rows_at(const RotArgs& a, int elem, int v) {
  for (const RotTensor& t : a.t) {
    if (t.H == 0) continue;
    if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) & (v * elem - 1)) return false;
    for (long long st : {t.xb, t.xs, t.xh, t.yb, t.ys, t.yh})
      if (st % v != 0) return false;
  }
  return true;
}

// The widest access that every run of columns, stride and base address allows: 16 bytes in ordinary use, down to
// one element for odd widths (a unit then moves V-fold less per index computation).
int pick_vec(const RotArgs& a, int elem) {
  const int run = a.plan.layout == UAA_ROTARY_HALF ? a.plan.rot / 2 : a.plan.rot;
  for (int v = 16 / elem; v > 1; v /= 2)
    if (run % v == 0 && (a.D - a.plan.rot) % v == 0 && rows_at(a, elem, v)) return v;
  return 1;
}

template <typename T>
int launch_t(RotArgs& a, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  const int v = pick_vec(a, sizeof(T));
  // Narrower accesses cost more than whole rows' detour: 40000 tokens, 24 + 8 heads of 64, bf16: 50 columns in halves
  // take 272 us by single elements and 122 by rows.  Where both move 16 bytes, the units are the faster (27280 x 80
  // heads of 128 in halves: 189 us, by rows 313).
  const bool rows = v < E && a.D % E == 0 && a.D / E <= 32 && rows_at(a, sizeof(T), E);
  a.pair_units = a.plan.layout == UAA_ROTARY_HALF || v == 1 ? a.plan.rot / 2 / v : a.plan.rot / v;
  a.units = rows ? a.D / E : a.pair_units + (a.D - a.plan.rot) / v;
  const uint32_t per_token = (a.t[0].H + a.t[1].H) * a.units;
  // a few units for every thread, as far as the angles fit
  uint32_t nt = 4 * kThreads / per_token;
  const uint32_t fit = a.plan.rot ? kMaxSmemPairs / (a.plan.rot / 2) : kMaxTokens;
  nt = nt > fit ? fit : nt;
  nt = nt > kMaxTokens ? kMaxTokens : nt;
  a.tokens_per_block = nt < 1 ? 1 : nt;
  // more blocks than fit at once, so that blocks end at different times (blocks of 256 threads: 247 us with 8 an SM, 189
  // with 64)
  const uint32_t need = (a.tokens - 1) / a.tokens_per_block + 1, cap = sm_count() * 128;
  const int grid = need < cap ? need : cap;
  const size_t smem = a.tokens_per_block * (a.plan.rot / 2) * sizeof(float2);
  if (rows) {
    if (a.plan.layout == UAA_ROTARY_HALF)
      rotary_rows_kernel<T, true><<<grid, kThreads, smem, s>>>(a);
    else
      rotary_rows_kernel<T, false><<<grid, kThreads, smem, s>>>(a);
    return check_launch("uaa_rotary");
  }
  switch (v) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch_v<T, 8>(a, grid, smem, s);
    case 4:
      return launch_v<T, 4>(a, grid, smem, s);
    case 2:
      return launch_v<T, 2>(a, grid, smem, s);
    default:
      return launch_v<T, 1>(a, grid, smem, s);
  }
}

int check_tensor(const char* fn, const char* name, const RotTensor& t, const RotArgs& a, int elem) {
  if (t.H == 0 || a.tokens == 0) return UAA_OK;
  if (!t.x || !t.y) return set_error(UAA_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) & (elem - 1))
    return set_error(UAA_ERR_INVALID_ARG, "%s: %s is not aligned to its element", fn, name);
  for (long long st : {t.xb, t.xs, t.xh, t.yb, t.ys, t.yh})
    if (st < 0 || st > (1LL << 40)) return set_error(UAA_ERR_INVALID_ARG, "%s: %s has a bad stride", fn, name);
  // output rows that overlap would be written by two threads: from the smallest stride up, each has to
  // step over everything that the smaller ones span
  struct Dim {
    long long stride, n;
  } d[3] = {{t.yb, a.B}, {t.ys, a.S}, {t.yh, t.H}};
  std::sort(d, d + 3, [](const Dim& u, const Dim& v) { return u.stride < v.stride; });
  long long span = a.D;
  for (const Dim& u : d) {
    if (u.n < 2) continue;
    if (u.stride < span) return set_error(UAA_ERR_INVALID_ARG, "%s: the rows of %s's output overlap", fn, name);
    span += u.stride * (u.n - 1);
  }
  return UAA_OK;
}

// Do the rows at p (strides b, s, h over nb, ns, nh) and at q, of D elements each, share an element?  Decided exactly where
// the strides are alike, as those of slices of one packed tensor are: then the distance of the two bases has to be a sum
// of strides, within a row.  Rows of other strides are only known to meet where they begin at one place.
struct Rows {
  const void* at;
  long long b, s, h;
  int nh;
};
bool rows_meet(const Rows& p, const Rows& q, int B, int S, int D, int elem) {
  const long long bytes = static_cast<const char*>(p.at) - static_cast<const char*>(q.at);
  if (bytes == 0) return true;
  struct Dim {
    long long stride;
    int n, m;
  } d[3] = {{p.b, B, B}, {p.s, S, S}, {p.h, p.nh, q.nh}};
  const long long other[3] = {q.b, q.s, q.h};
  auto span = [&](const Rows& r) { return ((B - 1) * r.b + (S - 1) * r.s + (r.nh - 1) * r.h + D) * elem; };
  if (bytes >= span(q) || -bytes >= span(p)) return false;
  for (int i = 0; i < 3; ++i) {
    if (d[i].n < 2) d[i].stride = other[i];
    if (d[i].n < 2 && d[i].m < 2) d[i].stride = 0;
    if (d[i].stride != other[i] && d[i].m > 1) return false;
  }
  std::sort(d, d + 3, [](const Dim& u, const Dim& v) { return u.stride > v.stride; });
  // the steps of each stride from the largest down: what is left is less than one of them, on either side
  for (int choice = 0; choice < 8; ++choice) {
    long long left = bytes;
    bool fits = true;
    for (int i = 0; i < 3 && fits; ++i) {
      if (d[i].stride == 0) continue;
      const long long st = d[i].stride * elem;
      long long k = left / st - (left % st < 0);  // rounded down
      k += choice >> i & 1;
      left -= k * st;
      fits = -k < d[i].n && k < d[i].m;  // row i of p lies where row i + k of q does
    }
    if (fits && left > -(long long)D * elem && left < (long long)D * elem) return true;
  }
  return false;
}

// An output may lie on its own input, row on row; on nothing else.
int check_overlap(const char* fn, const RotArgs& a, int elem) {
  const char* names[2] = {"q", "k"};
  auto in = [&](const RotTensor& t) { return Rows{t.x, t.xb, t.xs, t.xh, t.H}; };
  auto out = [&](const RotTensor& t) { return Rows{t.y, t.yb, t.ys, t.yh, t.H}; };
  for (int i = 0; i < 2; ++i) {
    const RotTensor& t = a.t[i];
    if (t.H == 0) continue;
    const bool in_place = t.x == t.y && (a.B < 2 || t.xb == t.yb) && (a.S < 2 || t.xs == t.ys) &&
                          (t.H < 2 || t.xh == t.yh);
    if (!in_place && rows_meet(out(t), in(t), a.B, a.S, a.D, elem))
      return set_error(UAA_ERR_INVALID_ARG, "%s: %s's output overlaps its input", fn, names[i]);
    const RotTensor& o = a.t[1 - i];
    if (o.H == 0) continue;
    if (rows_meet(out(t), in(o), a.B, a.S, a.D, elem))
      return set_error(UAA_ERR_INVALID_ARG, "%s: %s's output overlaps %s", fn, names[i], names[1 - i]);
    if (rows_meet(out(t), out(o), a.B, a.S, a.D, elem))
      return set_error(UAA_ERR_INVALID_ARG, "%s: the outputs of q and k overlap", fn);
  }
  return UAA_OK;
}

int check_plan(const char* fn, const uaa_rotary_plan* p, int D) {
  if (!p) return set_error(UAA_ERR_INVALID_ARG, "%s: the plan is NULL", fn);
  if (p->rot < 0 || p->rot % 2 || p->rot > 2 * kMaxPairs || p->rot > D)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d rotated columns of a head of %d", fn, p->rot, D);
  if (p->layout != UAA_ROTARY_HALF && p->layout != UAA_ROTARY_INTERLEAVED)
    return set_error(UAA_ERR_INVALID_ARG, "%s: layout %d", fn, p->layout);
  if (p->axes < 1 || p->axes > UAA_ROTARY_MAX_AXES) return set_error(UAA_ERR_INVALID_ARG, "%s: %d axes", fn, p->axes);
  for (int i = 0; i < p->rot / 2; ++i)
    if (p->axis[i] >= p->axes) return set_error(UAA_ERR_INVALID_ARG, "%s: pair %d follows axis %d", fn, i, p->axis[i]);
  if (!isfinite(p->magnitude)) return set_error(UAA_ERR_INVALID_ARG, "%s: the magnitude is not finite", fn);
  return UAA_OK;
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" int uaa_rotary_plan_init(uaa_rotary_plan* plan, int layout, int axes, const int* widths, double base,
                                    int scaling, double factor, double original, double alpha, double beta) {
  const char* fn = "uaa_rotary_plan_init";
  if (!plan || !widths) return set_error(UAA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (layout != UAA_ROTARY_HALF && layout != UAA_ROTARY_INTERLEAVED)
    return set_error(UAA_ERR_INVALID_ARG, "%s: layout %d", fn, layout);
  if (axes < 1 || axes > UAA_ROTARY_MAX_AXES)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d axes (1..%d)", fn, axes, UAA_ROTARY_MAX_AXES);
  if (!(base >= 1.0) || !isfinite(base)) return set_error(UAA_ERR_INVALID_ARG, "%s: base must be >= 1", fn);
  if (scaling < UAA_ROTARY_NONE || scaling > UAA_ROTARY_PARTS)
    return set_error(UAA_ERR_INVALID_ARG, "%s: scaling %d", fn, scaling);
  if (scaling != UAA_ROTARY_NONE && (!(factor >= 1.0) || !isfinite(factor)))
    return set_error(UAA_ERR_INVALID_ARG, "%s: the scaling factor must be >= 1", fn);
  if (scaling == UAA_ROTARY_PARTS && (!(original > 0.0) || !isfinite(original) || !(alpha >= 0.0) ||
                                      !(beta > alpha) || !isfinite(beta)))
    return set_error(UAA_ERR_INVALID_ARG, "%s: by parts needs original > 0 and 0 <= alpha < beta", fn);
  uaa_rotary_plan p{};
  p.layout = layout;
  p.axes = axes;
  p.magnitude = scaling == UAA_ROTARY_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  const double two_pi = 6.283185307179586476925;
  for (int x = 0; x < axes; ++x) {
    const int w = widths[x];
    if (w < 0 || w % 2 || w > 2 * kMaxPairs || p.rot + w > 2 * kMaxPairs)
      return set_error(UAA_ERR_INVALID_ARG, "%s: axis %d has %d columns (even, %d in all at most)", fn, x, w,
                       2 * kMaxPairs);
    double b = base;
    if (scaling == UAA_ROTARY_NTK && w > 2) b *= pow(factor, w / (w - 2.0));
    for (int j = 0; j < w / 2; ++j) {
      double f = pow(b, -2.0 * j / w);  // radians per position
      if (scaling == UAA_ROTARY_LINEAR) f /= factor;
      if (scaling == UAA_ROTARY_PARTS) {
        double keep = (original * f / two_pi - alpha) / (beta - alpha);
        keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
        f = keep * f + (1.0 - keep) * f / factor;
      }
      const int i = p.rot / 2 + j;
      p.turns[i] = static_cast<uint64_t>(ldexp(f / two_pi, 64) + 0.5);  // f <= 1: below 2^62
      p.axis[i] = static_cast<uint8_t>(x);
    }
    p.rot += w;
  }
  *plan = p;
  return UAA_OK;
}

extern "C" int uaa_rotary(const uaa_rotary_plan* plan, const uaa_rotary_tensor* q, const uaa_rotary_tensor* k,
                          const void* positions, int pos64, long long pos_batch_stride, long long pos_token_stride,
                          long long start, int B, int S, int D, int dtype, int inverse, uaa_stream_t stream) {
  const char* fn = "uaa_rotary";
  if (!q) return set_error(UAA_ERR_INVALID_ARG, "%s: q is NULL", fn);
  if (B < 0 || S < 0 || D < 1 || q->H < 0 || (k && k->H < 0))
    return set_error(UAA_ERR_INVALID_ARG, "%s: bad sizes B=%d S=%d D=%d", fn, B, S, D);
  if (D > 65536 || q->H > 65535 || (k && k->H > 65535))
    return set_error(UAA_ERR_UNSUPPORTED, "%s: D must be <= 65536 and the heads <= 65535", fn);
  if (dtype != UAA_BF16 && dtype != UAA_FP16 && dtype != UAA_FP32)
    return set_error(UAA_ERR_INVALID_ARG, "%s: dtype %d", fn, dtype);
  int st = check_plan(fn, plan, D);
  if (st) return st;
  if ((long long)B * S >= (1LL << 31)) return set_error(UAA_ERR_UNSUPPORTED, "%s: B*S must be below 2^31", fn);
  RotArgs a{};
  auto take = [&](const uaa_rotary_tensor& t) {
    return RotTensor{t.x, t.y, t.x_batch, t.x_token, t.x_head, t.y_batch, t.y_token, t.y_head, t.H,
                     (B - 1) * t.y_batch + (S - 1) * t.y_token + (t.H - 1) * t.y_head + D};
  };
  a.t[0] = take(*q);
  if (k) a.t[1] = take(*k);
  a.positions = positions;
  a.pos64 = pos64;
  a.pb = pos_batch_stride;
  a.ps = pos_token_stride;
  a.start = start;
  a.B = B;
  a.S = S;
  a.D = D;
  a.inverse = inverse;
  a.tokens = static_cast<uint32_t>((long long)B * S);
  a.plan = *plan;
  const int elem = dtype == UAA_FP32 ? 4 : 2;
  if ((st = check_tensor(fn, "q", a.t[0], a, elem)) || (st = check_tensor(fn, "k", a.t[1], a, elem))) return st;
  if (a.tokens && (st = check_overlap(fn, a, elem))) return st;
  if (positions && (reinterpret_cast<uintptr_t>(positions) & (pos64 ? 7 : 3)))
    return set_error(UAA_ERR_INVALID_ARG, "%s: positions are not aligned to their element", fn);
  if (a.tokens == 0 || a.t[0].H + a.t[1].H == 0) return UAA_OK;
  // a unit index of a block is 32 bits
  if ((long long)(a.t[0].H + a.t[1].H) * D * kMaxTokens >= (1LL << 31))
    return set_error(UAA_ERR_UNSUPPORTED, "%s: a token's heads hold too many columns", fn);
  if ((st = get_check_ctx(&a.ctx))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == UAA_BF16) return launch_t<__nv_bfloat16>(a, s);
  if (dtype == UAA_FP16) return launch_t<__half>(a, s);
  return launch_t<float>(a, s);
}
