// Attention over packed sequences and over the pages of a cache, forward (the
// formulas stand in seq_shared.cuh).  One warp per (token, query head): the keys
// one after the other, a running maximum and sum.
#include <float.h>

#include "seq_shared.cuh"

namespace uaa {
namespace {

template <int D, bool kPaged>
__global__ void __launch_bounds__(256) seq_fwd_rows_kernel(const __grid_constant__ SeqArgs a, DevCtx ctx) {
  const uaa_seqs& s = a.s;
  constexpr int P = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)s.T * s.Hq;
  const int fp16 = s.dtype == UAA_FP16;
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
    const int t = (int)(r / s.Hq), h = (int)(r % s.Hq), hk = h / a.g;
    const int b = seq_of_token(s.starts, s.B, t);
    if (b < 0) continue;  // behind the last sequence: left as it was
    const Seq q = load_seq<kPaged>(s, b);
    if (q.bad && lane == 0) atomicOr(ctx.status, kStatusBadPage);
    const int keys = keys_of(s, q, t - q.q0);
    float x[P], acc[P], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = load16(s.q, (size_t)t * s.q_row + (size_t)h * s.q_head + lane * P + i, fp16) * (s.scale * kLog2e);
      acc[i] = 0.f;
    }
    for (int j = 0; j < keys; ++j) {
      size_t ka, va;
      if constexpr (kPaged) {
        const int page = s.table[(size_t)q.k0 * s.width + j / s.page], at = j % s.page;
        if (page < 0 || page >= s.pages) {
          if (lane == 0) atomicOr(ctx.status, kStatusBadPage);
          continue;
        }
        ka = (size_t)page * s.k_page + (size_t)at * s.k_row;
        va = (size_t)page * s.v_page + (size_t)at * s.v_row;
      } else {
        ka = (size_t)(q.k0 + j) * s.k_row;
        va = (size_t)(q.k0 + j) * s.v_row;
      }
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i) d += x[i] * load16(s.k, ka + (size_t)hk * s.k_head + lane * P + i, fp16);
#pragma unroll
      for (int o = 16; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
      if (d > top) {
        const float now = fminf(d, FLT_MAX);  // finite: a score of +inf then gives p = sum = +inf and NaN behind it
        const float f = exp2f(top - now);
        sum *= f;
#pragma unroll
        for (int i = 0; i < P; ++i) acc[i] *= f;
        top = now;
      }
      const float p = d == -INFINITY ? 0.f : exp2f(d - top);
      sum += p;
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] += p * load16(s.v, va + (size_t)hk * s.v_head + lane * P + i, fp16);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) store16(s.out, (size_t)r * D + lane * P + i, sum == 0.f ? 0.f : acc[i] / sum, fp16);
    if (lane == 0) s.lse[(size_t)h * s.T + t] = sum == 0.f ? -INFINITY : (top + log2f(sum)) / kLog2e;
  }
}

size_t workspace_bytes(int T, int g, int D) {
  (void)T, (void)g, (void)D;
  return 256;
}

template <bool kPaged>
int seq_fwd(const char* fn, const uaa_seqs* s, void* workspace, size_t bytes, cudaStream_t stream) {
  int st = check_seqs(fn, s, kPaged);
  if (st) return st;
  if (s->T == 0 || s->B == 0) return UAA_OK;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  const size_t need = workspace_bytes(s->T, s->Hq / s->Hk, s->D);
  if (bytes < need) return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, bytes, need);
  DevCtx ctx;
  if ((st = get_dev_ctx(&ctx))) return st;
  const SeqArgs a = seq_args(*s);
  const long long blocks = ((long long)s->T * s->Hq + 7) / 8;
  const int grid = (int)(blocks < 152 * 8 ? blocks : 152 * 8);
  if (s->D == 64) seq_fwd_rows_kernel<64, kPaged><<<grid, 256, 0, stream>>>(a, ctx);
  else seq_fwd_rows_kernel<128, kPaged><<<grid, 256, 0, stream>>>(a, ctx);
  return check_launch(fn);
}

}  // namespace
}  // namespace uaa

extern "C" size_t uaa_attn_seqs_workspace_bytes(int T, int Hq, int Hk, int D) {
  if (T < 0 || Hk < 1 || Hq < 1 || Hq % Hk || (D != 64 && D != 128)) return 0;
  return uaa::workspace_bytes(T, Hq / Hk, D);
}

extern "C" int uaa_attn_packed_fwd(const uaa_seqs* args, void* workspace, size_t workspace_bytes, uaa_stream_t stream) {
  return uaa::seq_fwd<false>("uaa_attn_packed_fwd", args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int uaa_attn_paged_fwd(const uaa_seqs* args, void* workspace, size_t workspace_bytes, uaa_stream_t stream) {
  return uaa::seq_fwd<true>("uaa_attn_paged_fwd", args, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
