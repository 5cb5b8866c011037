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
// Codes are exact: code = rint(x * (127 / top)) in 32 bits unless that product
// lies within 2^-15 of a border between two codes (its error is below 127 * 2^-22
// of a code); there 254 |x| and (2 k + 1) top are compared, which are exact in 64
// bits.  A row with an infinity or a NaN gets a NaN step and comes back as NaN,
// so a run that diverged still shows it.  A row whose top is below 2^-119 (where
// 127 / top would overflow) is stored as zeros.
//
// Bound: HBM, one pass each way.  A lane holds 16 consecutive values of a row in
// registers (16 bytes of codes), a group of G lanes (G the power of two that
// covers the row) finds the top with shuffles.
#include <cuda_fp16.h>
#include <math.h>

#include "uaa_common.cuh"

namespace uaa {
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
};

__device__ __forceinline__ void read16(const float* p, float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + i);
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ float2 widen(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 widen(__half2 v) { return __half22float2(v); }
template <typename T2>
__device__ __forceinline__ void read16_2(const void* p, float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer / 8; ++i) {
    const uint4 a = __ldcs(static_cast<const uint4*>(p) + i);
    const T2* h = reinterpret_cast<const T2*>(&a);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = widen(h[e]);
      v[8 * i + 2 * e] = f.x, v[8 * i + 2 * e + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void read16(const __nv_bfloat16* p, float (&v)[kPer]) { read16_2<__nv_bfloat162>(p, v); }
__device__ __forceinline__ void read16(const __half* p, float (&v)[kPer]) { read16_2<__half2>(p, v); }

__device__ __forceinline__ void write16(float* p, const float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer / 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
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
__device__ __forceinline__ void write16(T* p, const float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer / 8; ++i)
    __stcs(reinterpret_cast<uint4*>(p) + i,
           make_uint4(narrow(p, v[8 * i], v[8 * i + 1]), narrow(p, v[8 * i + 2], v[8 * i + 3]),
                      narrow(p, v[8 * i + 4], v[8 * i + 5]), narrow(p, v[8 * i + 6], v[8 * i + 7])));
}

__device__ __forceinline__ int tensor_of(const ActArgs& a, long long row) {
  int t = 0;
#pragma unroll 1
  while (t + 1 < a.n && row >= a.first[t + 1]) ++t;
  return t;
}

// round(127 x / top) where t = x * (127 / top) in 32 bits is within 2^-15 of k + 1/2
__device__ __noinline__ float border_code(float x, float top, float t) {
  const double k = floor(fabs(static_cast<double>(t)));  // the lower of the two codes
  const double d = 254.0 * fabs(static_cast<double>(x)) - (2.0 * k + 1.0) * static_cast<double>(top);
  const bool odd = static_cast<int>(k) & 1;
  const double c = d > 0.0 || (d == 0.0 && odd) ? k + 1.0 : k;
  return copysignf(static_cast<float>(c), x);
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) act8_pack_kernel(const __grid_constant__ ActArgs a) {
  const int lane = threadIdx.x % G;
  const bool active = lane * kPer < a.D;
  const long long rows = a.first[a.n], stride = (long long)gridDim.x * (kThreads / G);
  // whole warps stay together for the shuffles: a group past the last row works on nothing
  const long long last = (rows + 32 / G - 1) / (32 / G) * (32 / G);
  for (long long r = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < last; r += stride) {
    const bool here = active && r < rows;
    const int t = r < rows ? tensor_of(a, r) : 0;
    const long long row = r - a.first[t], at = row * a.D + lane * kPer;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = 0.f;
    if (here) read16(static_cast<const T*>(a.x[t]) + at, v);
    uint32_t top_bits = 0;  // magnitudes as integers: infinities and NaN are the largest
#pragma unroll
    for (int i = 0; i < kPer; ++i) top_bits = max(top_bits, __float_as_uint(v[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = G / 2; o > 0; o /= 2) top_bits = max(top_bits, __shfl_xor_sync(0xffffffffu, top_bits, o));
    const float top = __uint_as_float(top_bits);
    const bool finite = top_bits < 0x7f800000u, some = top >= 0x1p-119f;
    const float inv = finite && some ? 127.f / top : 0.f;
    uint32_t packed[4] = {0u, 0u, 0u, 0u};
    if (inv > 0.f) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float u = v[i] * inv;
        float c = rintf(u);
        if (fabsf(u - c) > 0.5f - 0x1p-15f) c = border_code(v[i], top, u);
        packed[i / 4] |= (static_cast<uint32_t>(static_cast<int>(c)) & 0xffu) << (8 * (i % 4));
      }
    }
    if (here) {
      __stcs(reinterpret_cast<uint4*>(a.codes[t] + at), make_uint4(packed[0], packed[1], packed[2], packed[3]));
      if (lane == 0) a.steps[t][row] = !finite ? __uint_as_float(0x7fc00000u) : some ? __fdiv_rz(top, 127.f) : 0.f;
    }
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(const __grid_constant__ ActArgs a) {
  const int lane = threadIdx.x % G;
  if (lane * kPer >= a.D) return;
  const long long rows = a.first[a.n], stride = (long long)gridDim.x * (kThreads / G);
  for (long long r = (long long)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < rows; r += stride) {
    const int t = tensor_of(a, r);
    const long long row = r - a.first[t], at = row * a.D + lane * kPer;
    const uint4 p = __ldcs(reinterpret_cast<const uint4*>(a.codes[t] + at));
    const float step = a.steps[t][row];
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      v[i] = static_cast<float>(static_cast<int8_t>(w[i / 4] >> (8 * (i % 4)))) * step;
    write16(static_cast<T*>(a.y[t]) + at, v);
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
  const long long need = (a.first[a.n] + kThreads / G - 1) / (kThreads / G), cap = (long long)sm_count() * 8;
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
