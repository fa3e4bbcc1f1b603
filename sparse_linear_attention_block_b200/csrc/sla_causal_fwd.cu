// Causal softmax attention of packed sequences with grouped heads, forward.
//
//   s_ab = scale q_a . k_b  (b <= a + Lk - Lq),  lse_a = log sum_b exp s_ab,
//   o_a = sum_b exp(s_ab - lse_a) v_b
//
// One warp per (query row, head); the features lie across the lanes and the
// running maximum and sum of the softmax in registers (fp32).
#include "sla_causal.h"
#include "sla_ptx.cuh"

namespace sla {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) causal_fwd_kernel(
    RowView q, RowView k, RowView v, const Seq* __restrict__ seqs, RowOut o,
    float* __restrict__ lse, int total_q, int G, float scale) {
  constexpr int E = D / 32;
  const Seq sq = seqs[blockIdx.x];
  const int h = blockIdx.y, lane = lane_id();
  for (int a = blockIdx.z * kWarps + threadIdx.x / 32; a < sq.nq; a += gridDim.z * kWarps) {
    float x[E], acc[E], m = -INFINITY, l = 0.f;
    const size_t row = size_t(sq.q0) + a;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = __bfloat162float(q.p[row * q.row + h * q.head + lane * E + e]);
      acc[e] = 0.f;
    }
    const int n = min(sq.nk, a + 1 + sq.nk - sq.nq);
    for (int b = 0; b < n; ++b) {
      const size_t kr = size_t(sq.k0) + b;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e)
        s += x[e] * __bfloat162float(k.p[kr * k.row + h / G * k.head + lane * E + e]);
      s = warp_sum(s) * scale;
      const float mn = fmaxf(m, s), c = __expf(m - mn), w = __expf(s - mn);
      l = l * c + w;
      m = mn;
#pragma unroll
      for (int e = 0; e < E; ++e)
        acc[e] = acc[e] * c + w * __bfloat162float(v.p[kr * v.row + h / G * v.head + lane * E + e]);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o.p[row * o.row + h * o.head + lane * E + e] = __float2bfloat16(acc[e] * inv);
    if (lane == 0) lse[size_t(h) * total_q + row] = l > 0.f ? m + logf(l) : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_causal_fwd(const CausalProblem& p, const void* q, const void* k, const void* v,
                              const Seq* seqs, void* o, float* lse, int* err, cudaStream_t s) {
  (void)err;
  using B = __nv_bfloat16;
  const RowView vq{static_cast<const B*>(q), p.q.row, p.q.head},
      vk{static_cast<const B*>(k), p.k.row, p.k.head},
      vv{static_cast<const B*>(v), p.v.row, p.v.head};
  const RowOut vo{static_cast<B*>(o), p.o.row, p.o.head};
  const int z = p.max_q < 64 * kWarps ? (p.max_q + kWarps - 1) / kWarps : 64;
  const dim3 grid(p.n_seq, p.Hq, z);
  if (p.d == 128)
    causal_fwd_kernel<128><<<grid, kWarps * 32, 0, s>>>(vq, vk, vv, seqs, vo, lse, p.total_q, p.G,
                                                        p.scale);
  else
    causal_fwd_kernel<64><<<grid, kWarps * 32, 0, s>>>(vq, vk, vv, seqs, vo, lse, p.total_q, p.G,
                                                       p.scale);
  return cudaGetLastError();
}

}  // namespace sla
