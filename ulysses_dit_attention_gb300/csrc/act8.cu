// Activation checkpoints in 8 bits: what a layer keeps between its forward and
// its backward pass, as signed 8-bit codes with one 32-bit step per row of D
// values, several tensors in one launch.
//
//   top = max |x|,  step = top / 127,  code = round(127 x / top) (ties to even),
//   value = code * step, rounded to the tensor's type when it is taken back.
//
// A row of N(0, 1) values has its top near 2.7, so the error of a value is
// uniform within half a step of 0.021: 0.6 % of the row's rms, against 2.6 % for
// an 8-bit float with three mantissa bits.
//
// Codes are exact.  code = rint(u), u = x * (127 / top) in 32 bits, whose error is
// below u * 2^-22.
//  * 32-bit and fp16 values: where u lies within 2^-15 of a border between two
//    codes, 254 |x| and (2 k + 1) top are compared, which are exact in 64 bits.
//  * bf16 values need no such test.  With x = X 2^(-s) and top = T in units of the
//    top's last bit (128 <= X, T <= 255), u is |254 X - (2 k + 1) T 2^s| / (2 T 2^s)
//    codes from a border.  Where the numerator is not 0 that is at least
//    1 / (510 * 2^s), and u < 254 / 2^s: more than u's error.  Where it is 0, either
//    T = 254, and 127 / top and u are exact, or 127 divides 2 k + 1, so x is half the
//    top: 63.5, to the even 64, which a quotient 127 / top rounded upward gives.
//    (The test cost 170 us of 530 at the size below: a quarter of all rows hold
//    half their top.)
// A row with an infinity or a NaN gets a NaN step and comes back as NaN, so a run
// that diverged still shows it.  A row whose top is below 2^-119 (where 127 / top
// would overflow) is stored as zeros.
//
// Bound: HBM, one pass each way.  A group of G lanes (G the power of two that
// covers the row at 16 values a lane) holds a row in registers and finds the top
// with shuffles.  A lane's 16 values are runs of 16 bytes, one in each part of
// the row, so that the lanes of a warp read and write whole sectors side by side
// (16 consecutive values a lane, in two half-sector accesses, took 556 us to
// pack and 356 us to unpack four bf16 tensors of 27280 x 40 x 128; this takes 264
// and 238 us, 6.3 and 7.1 TB/s).  The grid holds 64 blocks a SM to pack and 1024
// to unpack: with 8, packing took 379 us (294 with 64, before the quotients below)
// and unpacking 276; with 1024 and 64, 316 and 249.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "uaa_common.cuh"

namespace uaa {

int validate_attn_sizes(const char* fn, int B, int Sq, int Sk, int H, int D, float scale);

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 16;  // values per lane

struct ActArgs {
  const void* x[UAA_ACT8_MAX_TENSORS];
  void* y[UAA_ACT8_MAX_TENSORS];
  int8_t* codes[UAA_ACT8_MAX_TENSORS];
  float* steps[UAA_ACT8_MAX_TENSORS];
  long long first[UAA_ACT8_MAX_TENSORS + 1];  // first row of each tensor, among all
  int n, D;
  DevCtx ctx;
};

// A lane's values: kRuns runs of kRun consecutive ones (16 bytes), run i at element i * (D / kRuns) + lane * kRun.
template <typename T>
struct Runs {
  static constexpr int kRun = 16 / sizeof(T), kRuns = kPer / kRun;
};

__device__ __forceinline__ void read_run(const float* p, float* v) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ float2 widen(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 widen(__half2 v) { return __half22float2(v); }
template <typename T2>
__device__ __forceinline__ void read_run2(const void* p, float* v) {
  const uint4 a = __ldcs(static_cast<const uint4*>(p));
  const T2* h = reinterpret_cast<const T2*>(&a);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = widen(h[e]);
    v[2 * e] = f.x, v[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ void read_run(const __nv_bfloat16* p, float* v) { read_run2<__nv_bfloat162>(p, v); }
__device__ __forceinline__ void read_run(const __half* p, float* v) { read_run2<__half2>(p, v); }

__device__ __forceinline__ void write_run(float* p, const float* v) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
}
__device__ __forceinline__ uint32_t narrow(__nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(__half*, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void write_run(T* p, const float* v) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(narrow(p, v[0], v[1]), narrow(p, v[2], v[3]), narrow(p, v[4], v[5]), narrow(p, v[6], v[7])));
}

__device__ __forceinline__ int tensor_of(const ActArgs& a, long long row) {
  int t = 0;
#pragma unroll 1
  while (t + 1 < a.n && row >= a.first[t + 1]) ++t;
  return t;
}

// round(127 x / top), ties to even, exactly: u = x * (127 / top) in 32 bits says between which two codes x lies.
__device__ __forceinline__ int exact_code(float x, float top, float u) {
  const double k = floor(fabs(static_cast<double>(u)));  // the lower of the two
  const double d = 254.0 * fabs(static_cast<double>(x)) - (2.0 * k + 1.0) * static_cast<double>(top);
  const int c = static_cast<int>(k);
  const int up = d > 0.0 || (d == 0.0 && (c & 1));
  return x < 0.f ? -(c + up) : c + up;
}

// top / 127 toward zero and 127 / top upward, exactly: a quotient q of 24 bits with one Newton step lies within half a
// last place and a little of the true one, the remainder fmaf(-q, d, n) is exact, and its sign says on which side; so
// the neighbour is the answer or q is.  (The directed divisions of the language, made for any operands, took 30 us of
// 294 at the size above.)
__device__ __forceinline__ float step_of(float top) {
  const float c = 1.f / 127.f;
  float q = top * c;
  q = fmaf(fmaf(-127.f, q, top), c, q);
  return fmaf(-127.f, q, top) < 0.f ? __uint_as_float(__float_as_uint(q) - 1u) : q;
}
__device__ __forceinline__ float inverse_of(float top) {
  if (top > 0x1p100f) return __fdiv_ru(127.f, top);  // 1 / top is no longer exact enough, or below the normal numbers
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(top));
  float q = 127.f * y;
  q = fmaf(fmaf(-q, top, 127.f), y, q);
  return fmaf(-q, top, 127.f) > 0.f ? __uint_as_float(__float_as_uint(q) + 1u) : q;
}

// (bf16: 32 registers, so that every thread of the SM holds a row's share in flight: 311 -> 295 us at the size above)
template <typename T, int G>
__global__ void __launch_bounds__(kThreads, std::is_same<T, __nv_bfloat16>::value ? 8 : 4)
    act8_pack_kernel(const __grid_constant__ ActArgs a) {
  constexpr int kRun = Runs<T>::kRun, kRuns = Runs<T>::kRuns;
  constexpr bool kBorders = !std::is_same<T, __nv_bfloat16>::value;
  const int lane = threadIdx.x % G;
  const bool active = lane * kPer < a.D;
  const int part = a.D / kRuns;
  const long long rows = a.first[a.n], stride = (long long)gridDim.x * (kThreads / G);
  // whole warps stay together for the shuffles: a group past the last row works on nothing
  const long long last = (rows + 32 / G - 1) / (32 / G) * (32 / G);
  for (long long r = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < last; r += stride) {
    const bool here = active && r < rows;
    const int t = here ? tensor_of(a, r) : 0;
    const long long row = r - a.first[t], at = row * a.D + lane * kRun;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.f;
    if (here) {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) read_run(static_cast<const T*>(a.x[t]) + at + i * part, v + i * kRun);
    }
    uint32_t top_bits = 0;  // magnitudes as integers: infinities and NaN are the largest
#pragma unroll
    for (int i = 0; i < kPer; ++i) top_bits = max(top_bits, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = G / 2; o > 0; o /= 2) top_bits = max(top_bits, __shfl_xor_sync(0xffffffffu, top_bits, o));
    const float top = __uint_as_float(top_bits);
    const bool finite = top_bits < 0x7f800000u, some = top >= 0x1p-119f;
    const float inv = finite && some ? inverse_of(top) : 0.f;
    uint32_t packed[4] = {0u, 0u, 0u, 0u};
    if (inv > 0.f) {
      const float2 inv2 = make_float2(inv, inv), magic = make_float2(12582912.f, 12582912.f);
      float off = 0.f;  // the furthest that a value lies from its code, in codes
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // adding 1.5 * 2^23 rounds to the nearest whole number, ties to even, and leaves it in the low bits
        const float2 u0 = mul2(make_float2(v[4 * i], v[4 * i + 1]), inv2), s0 = add2(u0, magic);
        const float2 u1 = mul2(make_float2(v[4 * i + 2], v[4 * i + 3]), inv2), s1 = add2(u1, magic);
        if (kBorders) {
          const float2 d0 = sub2(u0, sub2(s0, magic)), d1 = sub2(u1, sub2(s1, magic));
          off = fmaxf(fmaxf(off, fmaxf(fabsf(d0.x), fabsf(d0.y))), fmaxf(fabsf(d1.x), fabsf(d1.y)));
        }
        packed[i] = __byte_perm(__byte_perm(__float_as_uint(s0.x), __float_as_uint(s0.y), 0x0040),
                                __byte_perm(__float_as_uint(s1.x), __float_as_uint(s1.y), 0x0040), 0x5410);
      }
      if (kBorders && off > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float u = v[i] * inv;
          if (fabsf(u - rintf(u)) > 0.5f - 0x1p-15f)
            packed[i / 4] = (packed[i / 4] & ~(0xffu << (8 * (i % 4)))) |
                            ((static_cast<uint32_t>(exact_code(v[i], top, u)) & 0xffu) << (8 * (i % 4)));
        }
      }
    }
    if (here) {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        if (!guard_store(a.ctx, at + i * part, kRun, (a.first[t + 1] - a.first[t]) * a.D)) continue;
        int8_t* c = a.codes[t] + at + i * part;
        if constexpr (kRun == 8)
          __stcs(reinterpret_cast<uint2*>(c), make_uint2(packed[2 * i], packed[2 * i + 1]));
        else
          __stcs(reinterpret_cast<uint32_t*>(c), packed[i]);
      }
      if (lane == 0 && guard_store(a.ctx, row, 1, a.first[t + 1] - a.first[t]))
        a.steps[t][row] = !finite ? __uint_as_float(0x7fc00000u) : some ? step_of(top) : 0.f;
    }
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(const __grid_constant__ ActArgs a) {
  constexpr int kRun = Runs<T>::kRun, kRuns = Runs<T>::kRuns;
  const int lane = threadIdx.x % G;
  if (lane * kPer >= a.D) return;
  const int part = a.D / kRuns;
  const long long rows = a.first[a.n], stride = (long long)gridDim.x * (kThreads / G);
  for (long long r = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < rows; r += stride) {
    const int t = tensor_of(a, r);
    const long long row = r - a.first[t], at = row * a.D + lane * kRun;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int8_t* p = a.codes[t] + at + i * part;
      if constexpr (kRun == 8) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2*>(p));
        w[2 * i] = c.x, w[2 * i + 1] = c.y;
      } else {
        w[i] = __ldcs(reinterpret_cast<const uint32_t*>(p));
      }
    }
    const float step = a.steps[t][row];
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))) * step;
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (guard_store(a.ctx, at + i * part, kRun, (a.first[t + 1] - a.first[t]) * a.D))
        write_run(static_cast<T*>(a.y[t]) + at + i * part, v + i * kRun);
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess || n <= 0)
    return 148;
  return n;
}

template <typename T, int G>
int launch_g(const ActArgs& a, bool pack, cudaStream_t s) {
  const long long need = (a.first[a.n] + kThreads / G - 1) / (kThreads / G);
  const long long cap = (long long)sm_count() * (pack ? 64 : 1024);
  const int grid = (int)(need < cap ? need : cap);
  if (pack)
    act8_pack_kernel<T, G><<<grid, kThreads, 0, s>>>(a);
  else
    act8_unpack_kernel<T, G><<<grid, kThreads, 0, s>>>(a);
  return check_launch(pack ? "uaa_act8_pack" : "uaa_act8_unpack");
}

template <typename T>
int launch_t(const ActArgs& a, bool pack, cudaStream_t s) {
  const int lanes = a.D / kPer;
  if (lanes <= 1) return launch_g<T, 1>(a, pack, s);
  if (lanes <= 2) return launch_g<T, 2>(a, pack, s);
  if (lanes <= 4) return launch_g<T, 4>(a, pack, s);
  if (lanes <= 8) return launch_g<T, 8>(a, pack, s);
  if (lanes <= 16) return launch_g<T, 16>(a, pack, s);
  return launch_g<T, 32>(a, pack, s);
}

int act8(const char* fn, bool pack, int n, const void* const* x, int8_t* const* codes, float* const* steps,
         const long long* rows, int D, int dtype, uaa_stream_t stream) {
  if (n < 0 || n > UAA_ACT8_MAX_TENSORS)
    return set_error(UAA_ERR_INVALID_ARG, "%s: %d tensors (0..%d)", fn, n, UAA_ACT8_MAX_TENSORS);
  if (n > 0 && (!x || !codes || !steps || !rows)) return set_error(UAA_ERR_INVALID_ARG, "%s: NULL array", fn);
  if (D < 1) return set_error(UAA_ERR_INVALID_ARG, "%s: D=%d", fn, D);
  if (D % kPer || D > 32 * kPer)
    return set_error(UAA_ERR_UNSUPPORTED, "%s: D=%d (multiples of %d up to %d are built)", fn, D, kPer, 32 * kPer);
  if (dtype != UAA_BF16 && dtype != UAA_FP16 && dtype != UAA_FP32)
    return set_error(UAA_ERR_INVALID_ARG, "%s: dtype %d", fn, dtype);
  ActArgs a{};
  a.D = D;
  for (int i = 0; i < n; ++i) {
    if (rows[i] < 0 || rows[i] > (1LL << 40))
      return set_error(UAA_ERR_INVALID_ARG, "%s: tensor %d has %lld rows", fn, i, rows[i]);
    if (rows[i] == 0) continue;
    if (!x[i] || !codes[i] || !steps[i]) return set_error(UAA_ERR_INVALID_ARG, "%s: tensor %d is NULL", fn, i);
    if ((reinterpret_cast<uintptr_t>(x[i]) | reinterpret_cast<uintptr_t>(codes[i])) & 15u)
      return set_error(UAA_ERR_INVALID_ARG, "%s: tensor %d or its codes are not 16-byte aligned", fn, i);
    if (reinterpret_cast<uintptr_t>(steps[i]) & 3u)
      return set_error(UAA_ERR_INVALID_ARG, "%s: the steps of tensor %d are not 4-byte aligned", fn, i);
    a.x[a.n] = x[i];
    a.y[a.n] = const_cast<void*>(x[i]);
    a.codes[a.n] = codes[i];
    a.steps[a.n] = steps[i];
    a.first[a.n + 1] = a.first[a.n] + rows[i];
    ++a.n;
  }
  if (a.n == 0) return UAA_OK;
  if (int st = get_check_ctx(&a.ctx)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == UAA_BF16) return launch_t<__nv_bfloat16>(a, pack, s);
  if (dtype == UAA_FP16) return launch_t<__half>(a, pack, s);
  return launch_t<float>(a, pack, s);
}

}  // namespace
}  // namespace uaa

extern "C" int uaa_act8_pack(int n, const void* const* x, int8_t* const* codes, float* const* steps,
                             const long long* rows, int D, int dtype, uaa_stream_t stream) {
  return uaa::act8("uaa_act8_pack", true, n, x, codes, steps, rows, D, dtype, stream);
}

extern "C" int uaa_act8_unpack(int n, const int8_t* const* codes, const float* const* steps, void* const* y,
                               const long long* rows, int D, int dtype, uaa_stream_t stream) {
  return uaa::act8("uaa_act8_unpack", false, n, y, const_cast<int8_t* const*>(codes), const_cast<float* const*>(steps),
                   rows, D, dtype, stream);
}

extern "C" size_t uaa_attn_bwd_act8_workspace_bytes(int B, int Sq, int Sk, int H, int D) {
  if (B < 0 || Sq < 0 || Sk < 0 || H < 0 || (D != 64 && D != 128)) return 0;
  // q, k, v, out in bf16 (each B * S * H * D * 2 bytes, rounded up to 256), then the backward's own workspace
  const size_t q = ((size_t)B * Sq * H * D * 2 + 255) & ~(size_t)255, k = ((size_t)B * Sk * H * D * 2 + 255) & ~(size_t)255;
  return 2 * q + 2 * k + uaa_attn_bwd_workspace_bytes(B, Sq, H, D);
}

extern "C" int uaa_attn_bwd_act8(const int8_t* const* codes, const float* const* steps, const void* dout,
                                 const float* lse, const uint8_t* key_mask, void* dq, void* dk, void* dv, int B, int Sq,
                                 int Sk, int H, int D, float scale, void* workspace, size_t workspace_bytes,
                                 uaa_stream_t stream) {
  const char* fn = "uaa_attn_bwd_act8";
  int st = uaa::validate_attn_sizes(fn, B, Sq, Sk, H, D, scale);
  if (st) return st;
  if ((uint64_t)B * H == 0 || (uint64_t)Sq + Sk == 0) return UAA_OK;
  if (Sq == 0) return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: keys without queries (Sq = 0)", fn);
  if (!codes || !steps) return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: codes or steps is NULL", fn);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  const size_t need = uaa_attn_bwd_act8_workspace_bytes(B, Sq, Sk, H, D);
  if (workspace_bytes < need)
    return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  // the backward's other operands are checked before anything is launched
  for (const void* p : {dout, static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!p || (reinterpret_cast<uintptr_t>(p) & 15u))
      return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: dout, dq, dk or dv is NULL or not 16-byte aligned", fn);
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return uaa::set_error(UAA_ERR_INVALID_ARG, "%s: lse is NULL or not 4-byte aligned", fn);
  const long long rows[4] = {(long long)B * Sq * H, (long long)B * Sk * H, (long long)B * Sk * H, (long long)B * Sq * H};
  void* y[4];
  char* at = static_cast<char*>(workspace);
  for (int i = 0; i < 4; ++i) {
    y[i] = at;
    at += ((size_t)rows[i] * D * 2 + 255) & ~(size_t)255;
  }
  if ((st = uaa_act8_unpack(4, codes, steps, y, rows, D, UAA_BF16, stream))) return st;
  return uaa_attn_bwd_cross(y[0], y[1], y[2], y[3], dout, lse, key_mask, dq, dk, dv, B, Sq, Sk, H, D, scale, at,
                            workspace_bytes - (at - static_cast<char*>(workspace)), stream);
}
