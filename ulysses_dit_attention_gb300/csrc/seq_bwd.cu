// Attention over packed sequences, backward (the formulas stand in seq_shared.cuh).
// One warp per (token, query head) for dQ and Delta, one per (token, key head) for dK and dV.
#include "seq_shared.cuh"

namespace uaa {
namespace {

struct BwdArgs {
  SeqArgs a;
  const void* dout;
  void *dq, *dk, *dv;
  float* delta;  // (T, Hq)
};

template <int P>
__device__ __forceinline__ void row16(float (&x)[P], const void* p, size_t at, int lane) {
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = load16(p, at + lane * P + i, 0);
}
template <int P>
__device__ __forceinline__ float dot(const float (&x)[P], const float (&y)[P]) {
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) d += x[i] * y[i];
#pragma unroll
  for (int o = 16; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
  return d;
}

template <int D>
__global__ void __launch_bounds__(256) seq_bwd_dq_rows_kernel(const __grid_constant__ BwdArgs w) {
  const SeqArgs& a = w.a;
  const uaa_seqs& s = a.s;
  constexpr int P = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)s.T * s.Hq;
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
    const int t = (int)(r / s.Hq), h = (int)(r % s.Hq), hk = h / a.g;
    const int b = seq_of_token(s.starts, s.B, t);
    if (b < 0) continue;
    const Seq q = load_seq<false>(s, b);
    const int keys = keys_of(s, q, t - q.q0);
    float x[P], o[P], g[P], k[P], v[P], acc[P] = {};
    row16(x, s.q, (size_t)t * s.q_row + (size_t)h * s.q_head, lane);
    row16(o, s.out, (size_t)r * D, lane);
    row16(g, w.dout, (size_t)r * D, lane);
    const float delta = dot(o, g), lse = s.lse[(size_t)h * s.T + t];
    if (lane == 0) w.delta[r] = delta;
    for (int j = 0; j < keys && lse != -INFINITY; ++j) {
      row16(k, s.k, (size_t)(q.k0 + j) * s.k_row + (size_t)hk * s.k_head, lane);
      row16(v, s.v, (size_t)(q.k0 + j) * s.v_row + (size_t)hk * s.v_head, lane);
      const float ds = expf(dot(x, k) * s.scale - lse) * (dot(g, v) - delta);
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] += ds * k[i];
    }
#pragma unroll
    for (int i = 0; i < P; ++i) store16(w.dq, (size_t)r * D + lane * P + i, acc[i] * s.scale, 0);
  }
}

template <int D>
__global__ void __launch_bounds__(256) seq_bwd_dkdv_rows_kernel(const __grid_constant__ BwdArgs w) {
  const SeqArgs& a = w.a;
  const uaa_seqs& s = a.s;
  constexpr int P = D / 32;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)s.Tk * s.Hk;
  for (long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += (long long)gridDim.x * 8) {
    const int t = (int)(r / s.Hk), hk = (int)(r % s.Hk);
    const int b = seq_of_token(s.starts_k ? s.starts_k : s.starts, s.B, t);
    if (b < 0) continue;
    const Seq q = load_seq<false>(s, b);
    const int j = t - q.k0, first = s.causal ? max(0, j - (q.m - q.n)) : 0;
    float x[P], g[P], k[P], v[P], dk[P] = {}, dv[P] = {};
    row16(k, s.k, (size_t)t * s.k_row + (size_t)hk * s.k_head, lane);
    row16(v, s.v, (size_t)t * s.v_row + (size_t)hk * s.v_head, lane);
    for (int i = first; i < q.n; ++i)
      for (int h = hk * a.g; h < hk * a.g + a.g; ++h) {
        const int tq = q.q0 + i;
        row16(x, s.q, (size_t)tq * s.q_row + (size_t)h * s.q_head, lane);
        row16(g, w.dout, ((size_t)tq * s.Hq + h) * D, lane);
        const float p = expf(dot(x, k) * s.scale - s.lse[(size_t)h * s.T + tq]);
        const float ds = p * (dot(g, v) - w.delta[(size_t)tq * s.Hq + h]);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          dk[e] += ds * x[e];
          dv[e] += p * g[e];
        }
      }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      store16(w.dk, (size_t)r * D + lane * P + e, dk[e] * s.scale, 0);
      store16(w.dv, (size_t)r * D + lane * P + e, dv[e], 0);
    }
  }
}

template <int D>
int launch_bwd(const BwdArgs& w, cudaStream_t stream) {
  seq_bwd_dq_rows_kernel<D><<<152 * 8, 256, 0, stream>>>(w);
  if (int st = check_launch("uaa_attn_packed_bwd")) return st;
  seq_bwd_dkdv_rows_kernel<D><<<152 * 8, 256, 0, stream>>>(w);
  return check_launch("uaa_attn_packed_bwd");
}

}  // namespace
}  // namespace uaa

using namespace uaa;

extern "C" size_t uaa_attn_packed_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int D) {
  if (B < 0 || T < 0 || Hk < 1 || Hq < 1 || (D != 64 && D != 128)) return 0;
  return ((size_t)T * Hq * 4 + 255) & ~(size_t)255;
}

extern "C" int uaa_attn_packed_bwd(const uaa_seqs* s, const void* dout, void* dq, void* dk, void* dv, void* workspace,
                                   size_t workspace_bytes, uaa_stream_t stream) {
  const char* fn = "uaa_attn_packed_bwd";
  int st = check_seqs(fn, s, false, true);
  if (st) return st;
  if (s->dtype != UAA_BF16) return set_error(UAA_ERR_UNSUPPORTED, "%s: the backward is built for bf16", fn);
  if (s->B == 0 || (s->T == 0 && s->Tk == 0)) return UAA_OK;
  if (s->T > 0 && ((st = check_dev_ptr(fn, "dout", dout)) || (st = check_dev_ptr(fn, "dq", dq)))) return st;
  if (s->Tk > 0 && ((st = check_dev_ptr(fn, "dk", dk)) || (st = check_dev_ptr(fn, "dv", dv)))) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace is NULL or not 256-byte aligned", fn);
  const size_t need = uaa_attn_packed_bwd_workspace_bytes(s->B, s->T, s->Hq, s->Hk, s->D);
  if (workspace_bytes < need)
    return set_error(UAA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", fn, workspace_bytes, need);
  BwdArgs w{seq_args(*s), dout, dq, dk, dv, static_cast<float*>(workspace)};
  return s->D == 64 ? launch_bwd<64>(w, static_cast<cudaStream_t>(stream)) : launch_bwd<128>(w, static_cast<cudaStream_t>(stream));
}
