// Shared by the kernels of differential attention: every head has two softmax
// maps over the same keys and reads the values by their difference,
//   A_m = softmax(scale q_m k_m^T + bias)      (m = 1, 2; D/2 columns each)
//   O   = (A_1 - lambda_h A_2) V,   O2 = A_2 V (kept for the backward).
// With dA = dO V^T the gradients are
//   Delta_2 = dO . O2,  Delta_1 = dO . O + lambda Delta_2     (= A_m dA per row)
//   dS_1 = A_1 (dA - Delta_1),  dS_2 = -lambda A_2 (dA - Delta_2)
//   dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = (A_1 - lambda A_2)^T dO
//   dlambda_h = -sum_{b, i} Delta_2.
// Sums, softmax statistics and accumulators are 32-bit; what a matrix
// instruction reads (P, dS) is rounded to bf16, its operands' type.
#pragma once

#include <math.h>

#include "uaa_common.cuh"

namespace uaa {

int validate_attn_sizes(const char* fn, int B, int Sq, int Sk, int H, int D, float scale);
int check_dev_ptr(const char* fn, const char* name, const void* p);

namespace {

constexpr int kTile = 128;              // query rows and keys of a tile
constexpr int kChunkBytes = 128 * 128;  // 128 rows x 128 bytes: 64 columns of a tile, 128-byte swizzled

// 4-D tiled tensor store from shared memory (bulk-group completion; out-of-range rows of the box are not written).
__device__ __forceinline__ void tma_store_4d(const void* smem_src, const CUtensorMap* map, int c0, int c1, int c2,
                                             int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ float load_lambda(const void* lam, int bf16, int h) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(lam)[h]) : static_cast<const float*>(lam)[h];
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Byte offset of 16-column step kk of map m within a tile of D columns (one or two 64-column chunks).
template <int D>
__host__ __device__ constexpr uint32_t map_step(int m, int kk) {
  const int col = m * (D / 2) + 16 * kk;
  return (col / 64) * kChunkBytes + (col % 64) * 2;
}

__host__ __device__ __forceinline__ int tiles_of(int S) { return (S + kTile - 1) / kTile; }

// 16 columns of this thread's TMEM lane, then a wait for the store.
__device__ __forceinline__ void tmem_st16_bits(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8_bits(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
                                                cudaSuccess || n <= 0)
    return 148;
  return n;
}

int check_lambda(const char* fn, const void* lam, int dtype) {
  if (dtype != UAA_BF16 && dtype != UAA_FP32)
    return set_error(UAA_ERR_INVALID_ARG, "%s: lambda must be bf16 or fp32 (dtype %d)", fn, dtype);
  if (!lam) return set_error(UAA_ERR_INVALID_ARG, "%s: lambda is NULL", fn);
  if (reinterpret_cast<uintptr_t>(lam) & (dtype == UAA_BF16 ? 1u : 3u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: lambda is not aligned to its element", fn);
  return UAA_OK;
}

int check_lse(const char* fn, const void* lse) {
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: lse is NULL or not 4-byte aligned", fn);
  return UAA_OK;
}

}  // namespace
}  // namespace uaa
