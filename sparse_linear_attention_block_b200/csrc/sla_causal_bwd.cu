// Causal softmax attention of packed sequences with grouped heads, backward.
//
//   D_a = o_a . do_a,  P_ab = exp(s_ab - lse_a),  dS_ab = P_ab (do_a . v_b - D_a)
//   dq_a = scale sum_b dS_ab k_b
//   dk_b = scale sum_{h of the group, a} dS_ab q_a,  dv_b = sum_{h, a} P_ab do_a
//
// Two kernels, one over queries and one over keys, so that every sum has one
// owner: no atomics, equal inputs give equal bits.
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

template <int E>
__device__ __forceinline__ void load_row(float (&x)[E], const RowView& t, size_t row, int head) {
#pragma unroll
  for (int e = 0; e < E; ++e)
    x[e] = __bfloat162float(t.p[row * t.row + head * t.head + lane_id() * E + e]);
}
template <int E>
__device__ __forceinline__ void store_row(const float (&x)[E], const RowOut& t, size_t row,
                                          int head, float f) {
#pragma unroll
  for (int e = 0; e < E; ++e)
    t.p[row * t.row + head * t.head + lane_id() * E + e] = __float2bfloat16(x[e] * f);
}
template <int E>
__device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) s += x[e] * y[e];
  return warp_sum(s);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) causal_dvec_kernel(RowView o, RowView d_o,
                                                                  const int* __restrict__ count, const Item* __restrict__ items,
                                                                  float* __restrict__ dvec,
                                                                  int total_q) {
  if (int(blockIdx.x) >= *count) return;
  const Seq sq = items[blockIdx.x].s;
  const int t0 = items[blockIdx.x].tile * kRowTile;
  const int h = blockIdx.y;
  for (int a = t0 + threadIdx.x / 32; a < min(sq.nq, t0 + kRowTile); a += kWarps) {
    float x[D / 32], y[D / 32];
    load_row(x, o, size_t(sq.q0) + a, h);
    load_row(y, d_o, size_t(sq.q0) + a, h);
    const float s = dot(x, y);
    if (lane_id() == 0) dvec[size_t(h) * total_q + sq.q0 + a] = s;
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) causal_dq_kernel(
    RowView q, RowView k, RowView v, RowView d_o, const int* __restrict__ count, const Item* __restrict__ items,
    const float* __restrict__ lse, const float* __restrict__ dvec, RowOut dq, int total_q, int G,
    float scale) {
  constexpr int E = D / 32;
  if (int(blockIdx.x) >= *count) return;
  const Seq sq = items[blockIdx.x].s;
  const int t0 = items[blockIdx.x].tile * kRowTile;
  const int h = blockIdx.y;
  for (int a = t0 + threadIdx.x / 32; a < min(sq.nq, t0 + kRowTile); a += kWarps) {
    const size_t row = size_t(sq.q0) + a;
    float x[E], g[E], acc[E] = {};
    load_row(x, q, row, h);
    load_row(g, d_o, row, h);
    const float l = lse[size_t(h) * total_q + row], dd = dvec[size_t(h) * total_q + row];
    const int n = min(sq.nk, a + 1 + sq.nk - sq.nq);
    for (int b = 0; b < n; ++b) {
      float kk[E], vv[E];
      load_row(kk, k, size_t(sq.k0) + b, h / G);
      load_row(vv, v, size_t(sq.k0) + b, h / G);
      const float ds = __expf(dot(x, kk) * scale - l) * (dot(g, vv) - dd);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += ds * kk[e];
    }
    store_row(acc, dq, row, h, scale);
  }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) causal_dkv_kernel(
    RowView q, RowView k, RowView v, RowView d_o, const int* __restrict__ count, const Item* __restrict__ items,
    const float* __restrict__ lse, const float* __restrict__ dvec, RowOut dk, RowOut dv,
    int total_q, int G, float scale) {
  constexpr int E = D / 32;
  if (int(blockIdx.x) >= *count) return;
  const Seq sq = items[blockIdx.x].s;
  const int t0 = items[blockIdx.x].tile * kRowTile;
  const int hk = blockIdx.y;
  for (int b = t0 + threadIdx.x / 32; b < min(sq.nk, t0 + kRowTile); b += kWarps) {
    float kk[E], vv[E], ak[E] = {}, av[E] = {};
    load_row(kk, k, size_t(sq.k0) + b, hk);
    load_row(vv, v, size_t(sq.k0) + b, hk);
    for (int h = hk * G; h < (hk + 1) * G; ++h)
      for (int a = max(0, b - (sq.nk - sq.nq)); a < sq.nq; ++a) {
        const size_t row = size_t(sq.q0) + a;
        float x[E], g[E];
        load_row(x, q, row, h);
        load_row(g, d_o, row, h);
        const float p = __expf(dot(x, kk) * scale - lse[size_t(h) * total_q + row]);
        const float ds = p * (dot(g, vv) - dvec[size_t(h) * total_q + row]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          ak[e] += ds * x[e];
          av[e] += p * g[e];
        }
      }
    store_row(ak, dk, size_t(sq.k0) + b, hk, scale);
    store_row(av, dv, size_t(sq.k0) + b, hk, 1.f);
  }
}

RowView view(const void* p, const sla_strides& s) {
  return {static_cast<const __nv_bfloat16*>(p), s.row, s.head};
}
RowOut out(void* p, const sla_strides& s) { return {static_cast<__nv_bfloat16*>(p), s.row, s.head}; }

}  // namespace

cudaError_t launch_causal_dvec(const CausalProblem& p, const ItemList& list, const void* o,
                               const void* d_o, float* dvec, cudaStream_t s) {
  const dim3 grid(list.most, p.Hq);
  if (p.d == 128)
    causal_dvec_kernel<128><<<grid, kWarps * 32, 0, s>>>(view(o, p.o), view(d_o, p.o), list.count, list.items, dvec,
                                                         p.total_q);
  else
    causal_dvec_kernel<64><<<grid, kWarps * 32, 0, s>>>(view(o, p.o), view(d_o, p.o), list.count, list.items, dvec,
                                                        p.total_q);
  return cudaGetLastError();
}

cudaError_t launch_causal_dq(const CausalProblem& p, const void* q, const void* k, const void* v,
                             const ItemList& list, const void* d_o, const float* lse, const float* dvec,
                             void* dq, int* err, cudaStream_t s) {
  (void)err;
  const dim3 grid(list.most, p.Hq);
  if (p.d == 128)
    causal_dq_kernel<128><<<grid, kWarps * 32, 0, s>>>(view(q, p.q), view(k, p.k), view(v, p.v),
                                                       view(d_o, p.o), list.count, list.items, lse, dvec,
                                                       out(dq, p.q), p.total_q, p.G, p.scale);
  else
    causal_dq_kernel<64><<<grid, kWarps * 32, 0, s>>>(view(q, p.q), view(k, p.k), view(v, p.v),
                                                      view(d_o, p.o), list.count, list.items, lse, dvec,
                                                      out(dq, p.q), p.total_q, p.G, p.scale);
  return cudaGetLastError();
}

cudaError_t launch_causal_dkv(const CausalProblem& p, const void* q, const void* k, const void* v,
                              const ItemList& list, const void* d_o, const float* lse,
                              const float* dvec, void* dk, void* dv, int* err, cudaStream_t s) {
  (void)err;
  const dim3 grid(list.most, p.Hkv);
  if (p.d == 128)
    causal_dkv_kernel<128><<<grid, kWarps * 32, 0, s>>>(
        view(q, p.q), view(k, p.k), view(v, p.v), view(d_o, p.o), list.count, list.items, lse, dvec, out(dk, p.k),
        out(dv, p.v), p.total_q, p.G, p.scale);
  else
    causal_dkv_kernel<64><<<grid, kWarps * 32, 0, s>>>(
        view(q, p.q), view(k, p.k), view(v, p.v), view(d_o, p.o), list.count, list.items, lse, dvec, out(dk, p.k),
        out(dv, p.v), p.total_q, p.G, p.scale);
  return cudaGetLastError();
}

}  // namespace sla
