// Differential attention, backward (the formulas stand in diff_shared.cuh).
#include "diff_shared.cuh"

namespace uaa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The E consecutive columns of a row that one lane holds (a row is spread over a warp: lanes 0-15 hold map 1).
template <int E>
__device__ __forceinline__ void load_cols(const __nv_bfloat16* p, float (&v)[E]) {
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + e));
    v[e] = f.x;
    v[e + 1] = f.y;
  }
}
template <int E>
__device__ __forceinline__ void store_cols(__nv_bfloat16* p, const float (&v)[E], float c) {
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(p + e) = __floats2bfloat162_rn(v[e] * c, v[e + 1] * c);
}
template <int E>
__device__ __forceinline__ float dot_cols(const float (&a)[E], const float (&b)[E]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) s = fmaf(a[e], b[e], s);
  return s;
}
// sum over the 16 lanes of a map (every lane gets its own map's), or over the whole warp
__device__ __forceinline__ float map_sum(float s) {
#pragma unroll
  for (int o = 8; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
__device__ __forceinline__ float warp_sum(float s) {
  s = map_sum(s);
  return s + __shfl_xor_sync(0xffffffffu, s, 16);
}

// Row vectors of the backward: (B, H, tiles, 2 maps, 128)
__host__ __device__ __forceinline__ size_t row_at(size_t bh, int Sq, int m, int i) {
  return ((bh * tiles_of(Sq) + i / 128) * 2 + m) * 128 + i % 128;
}

// Delta_m and -LSE_m * log2(e) of every query row; rows past Sq get 0 and -inf (P = 0).
template <int D>
__global__ void __launch_bounds__(kThreads) diff_rows_kernel(
    const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ out2,
    const __nv_bfloat16* __restrict__ dout, const float* __restrict__ lse, const void* __restrict__ lam, int lam_bf16,
    float* __restrict__ delta, float* __restrict__ nl2, int B, int Sq, int H) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int pad = tiles_of(Sq) * 128;
  const size_t rows = (size_t)B * pad * H;
  for (size_t r = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += (size_t)gridDim.x * kWarps) {
    const int h = r % H, i = r / H % pad, b = r / H / pad;
    const size_t bh = (size_t)b * H + h;
    float d1 = 0.f, d2 = 0.f;
    if (i < Sq) {
      const size_t at = (((size_t)b * Sq + i) * H + h) * D + lane * E;
      float o[E], p[E], g[E];
      load_cols<E>(out + at, o);
      load_cols<E>(out2 + at, p);
      load_cols<E>(dout + at, g);
      d2 = warp_sum(dot_cols<E>(p, g));
      d1 = fmaf(load_lambda(lam, lam_bf16, h), d2, warp_sum(dot_cols<E>(o, g)));
    }
    if (lane < 2) {
      const float l = i < Sq ? lse[(bh * 2 + lane) * Sq + i] : -INFINITY;
      delta[row_at(bh, Sq, lane, i)] = lane ? d2 : d1;
      nl2[row_at(bh, Sq, lane, i)] = l == -INFINITY ? -INFINITY : -l * kLog2e;
    }
  }
}

// dlambda_h = -sum of Delta_2 over the head's rows, one block per head, in a fixed order.
__global__ void __launch_bounds__(1024) diff_dlambda_kernel(const float* __restrict__ delta, void* __restrict__ dlam,
                                                            int lam_bf16, int B, int Sq, int H) {
  __shared__ float part[32];
  const int h = blockIdx.x, tiles = tiles_of(Sq);
  float s = 0.f;
  for (int b = 0; b < B; ++b)
    for (int i = threadIdx.x; i < tiles * 128; i += blockDim.x) s += delta[row_at((size_t)b * H + h, Sq, 1, i)];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = warp_sum(part[threadIdx.x]);
    if (threadIdx.x == 0) {
      if (lam_bf16)
        static_cast<__nv_bfloat16*>(dlam)[h] = __float2bfloat16_rn(-s);
      else
        static_cast<float*>(dlam)[h] = -s;
    }
  }
}

// One warp per (b, h, query row): dQ.
template <int D>
__global__ void __launch_bounds__(kThreads) diff_dq_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    const __nv_bfloat16* __restrict__ dout, const void* __restrict__ lam, int lam_bf16,
    const float* __restrict__ delta, const float* __restrict__ nl2, const uint8_t* __restrict__ mask,
    __nv_bfloat16* __restrict__ dq, int B, int Sq, int Sk, int H, float scale, float scale_log2) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, m = lane >> 4;
  const size_t rows = (size_t)B * H * Sq;
  for (size_t r = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += (size_t)gridDim.x * kWarps) {
    const int i = r % Sq, h = r / Sq % H, b = r / Sq / H;
    const size_t at = (((size_t)b * Sq + i) * H + h) * D + lane * E, ra = row_at((size_t)b * H + h, Sq, m, i);
    const float w = m ? -load_lambda(lam, lam_bf16, h) : 1.f;
    float qv[E], g[E], acc[E] = {};
    load_cols<E>(q + at, qv);
    load_cols<E>(dout + at, g);
    for (int j = 0; j < Sk; ++j) {
      if (mask && !mask[(size_t)b * Sk + j]) continue;
      const size_t kat = (((size_t)b * Sk + j) * H + h) * D + lane * E;
      float kv[E], vv[E];
      load_cols<E>(k + kat, kv);
      load_cols<E>(v + kat, vv);
      const float p = exp2f(fmaf(map_sum(dot_cols<E>(qv, kv)), scale_log2, nl2[ra]));
      const float ds = w * p * (warp_sum(dot_cols<E>(g, vv)) - delta[ra]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(ds, kv[e], acc[e]);
    }
    store_cols<E>(dq + at, acc, scale);
  }
}

// One warp per (b, h, key row): dK and dV.
template <int D>
__global__ void __launch_bounds__(kThreads) diff_dkdv_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
    const __nv_bfloat16* __restrict__ dout, const void* __restrict__ lam, int lam_bf16,
    const float* __restrict__ delta, const float* __restrict__ nl2, const uint8_t* __restrict__ mask,
    __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv, int B, int Sq, int Sk, int H, float scale,
    float scale_log2) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, m = lane >> 4;
  const size_t rows = (size_t)B * H * Sk;
  for (size_t r = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5); r < rows; r += (size_t)gridDim.x * kWarps) {
    const int j = r % Sk, h = r / Sk % H, b = r / Sk / H;
    const size_t at = (((size_t)b * Sk + j) * H + h) * D + lane * E;
    const float w = m ? -load_lambda(lam, lam_bf16, h) : 1.f;
    float kv[E], vv[E], ak[E] = {}, av[E] = {};
    load_cols<E>(k + at, kv);
    load_cols<E>(v + at, vv);
    const int nq = !mask || mask[(size_t)b * Sk + j] ? Sq : 0;
    for (int i = 0; i < nq; ++i) {
      const size_t qat = (((size_t)b * Sq + i) * H + h) * D + lane * E, ra = row_at((size_t)b * H + h, Sq, m, i);
      float qv[E], g[E];
      load_cols<E>(q + qat, qv);
      load_cols<E>(dout + qat, g);
      const float p = w * exp2f(fmaf(map_sum(dot_cols<E>(qv, kv)), scale_log2, nl2[ra]));
      const float ds = p * (warp_sum(dot_cols<E>(g, vv)) - delta[ra]);
      const float both = p + __shfl_xor_sync(0xffffffffu, p, 16);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ak[e] = fmaf(ds, qv[e], ak[e]);
        av[e] = fmaf(both, g[e], av[e]);
      }
    }
    store_cols<E>(dk + at, ak, scale);
    store_cols<E>(dv + at, av, 1.f);
  }
}

int grid_for(size_t rows) {
  const size_t need = (rows + kWarps - 1) / kWarps, cap = (size_t)device_sms() * 8;
  return (int)(need < cap ? need : cap);
}

using bf = __nv_bfloat16;
const bf* in(const void* p) { return static_cast<const bf*>(p); }
bf* to(void* p) { return static_cast<bf*>(p); }

template <int D>
int launch_bwd(const void* q, const void* k, const void* v, const void* lam, int lam_bf16, const void* out,
               const void* out2, const void* dout, const float* lse, const uint8_t* mask, void* dq, void* dk, void* dv,
               void* dlam, int B, int Sq, int Sk, int H, float scale, float* delta, cudaStream_t s) {
  float* nl2 = delta + (size_t)B * H * tiles_of(Sq) * 256;
  int st;
  diff_rows_kernel<D><<<grid_for((size_t)B * H * tiles_of(Sq) * 128), kThreads, 0, s>>>(
      in(out), in(out2), in(dout), lse, lam, lam_bf16, delta, nl2, B, Sq, H);
  if ((st = check_launch("uaa_diff_attn_bwd (rows)"))) return st;
  diff_dlambda_kernel<<<H, 1024, 0, s>>>(delta, dlam, lam_bf16, B, Sq, H);
  if ((st = check_launch("uaa_diff_attn_bwd (dlambda)"))) return st;
  diff_dkdv_kernel<D><<<grid_for((size_t)B * H * Sk), kThreads, 0, s>>>(in(q), in(k), in(v), in(dout), lam, lam_bf16,
                                                                       delta, nl2, mask, to(dk), to(dv), B, Sq, Sk, H,
                                                                       scale, scale * kLog2e);
  if ((st = check_launch("uaa_diff_attn_bwd (dK/dV)"))) return st;
  diff_dq_kernel<D><<<grid_for((size_t)B * H * Sq), kThreads, 0, s>>>(in(q), in(k), in(v), in(dout), lam, lam_bf16,
                                                                     delta, nl2, mask, to(dq), B, Sq, Sk, H, scale,
                                                                     scale * kLog2e);
  return check_launch("uaa_diff_attn_bwd (dQ)");
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" size_t uaa_diff_attn_bwd_workspace_bytes(int B, int Sq, int H, int D) {
  if (B < 0 || Sq < 0 || H < 0 || (D != 64 && D != 128)) return 0;
  // Delta and -LSE*log2(e), each (B, H, tiles, 2, 128) fp32
  return (size_t)B * H * tiles_of(Sq) * 2048;
}

extern "C" int uaa_diff_attn_bwd(const void* q, const void* k, const void* v, const void* lambda, int lambda_dtype,
                                 const void* out, const void* out2, const void* dout, const float* lse,
                                 const uint8_t* key_mask, void* dq, void* dk, void* dv, void* dlambda, int B, int Sq,
                                 int Sk, int H, int D, float scale, void* workspace, size_t workspace_bytes,
                                 uaa_stream_t stream) {
  const char* fn = "uaa_diff_attn_bwd";
  int st = validate_attn_sizes(fn, B, Sq, Sk, H, D, scale);
  if (st) return st;
  if ((uint64_t)B * H == 0 || (uint64_t)Sq + Sk == 0) return UAA_OK;
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
  const size_t need = uaa_diff_attn_bwd_workspace_bytes(B, Sq, H, D);
  if (workspace_bytes < need)
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  auto go = D == 64 ? launch_bwd<64> : launch_bwd<128>;
  return go(q, k, v, lambda, lambda_dtype == UAA_BF16, out, out2, dout, lse, key_mask, dq, dk, dv, dlambda, B, Sq, Sk,
            H, scale, static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
}
