// Linear attention with a decay for each head, over packed sequences:
//   S_t = l S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  l = exp(log_decay)
//
// With do the gradient of o and B_t that of S_t (B_last includes d_state_out,
// B_t = l B_{t+1} + scale q_t do_t^T):
//   dq_t = scale S_t do_t,  dk_t = B_t v_t,  dv_t = B_t^T k_t,  d_state_in = l B_0
// so every output is the same recurrence with other inputs in the parts of
// query (x), key (y) and value (z), forward or from the last token on:
//   o:  x = q, y = k, z = v      dq: x = do, y = v, z = k (state transposed)
//   dv: x = k, y = q, z = do     dk: x = v, y = do, z = q, both reversed
#include "sla_causal.h"
#include "sla_ptx.cuh"

namespace sla {
namespace {

// One CTA per (sequence, head), one thread per column of the state (fp32).
template <int D>
__global__ void __launch_bounds__(D) decay_run_kernel(DecayRun r, const Seq* __restrict__ seqs,
                                                      const float* __restrict__ log_decay, int H,
                                                      float fs_out, float fs_up) {
  __shared__ float sx[D], sy[D];
  const Seq sq = seqs[blockIdx.x];
  if (sq.nq < 0) return;
  const int h = blockIdx.y, z = threadIdx.x;
  const Factor l = decay_factor(decay_checked(log_decay[h]), 1);
  float S[D];
  const size_t base = (size_t(blockIdx.x) * H + h) * D * D;
#pragma unroll
  for (int y = 0; y < D; ++y)
    S[y] = r.state_in ? r.state_in[base + (r.state_t ? z * D + y : y * D + z)] : 0.f;
  for (int i = 0; i < sq.nq; ++i) {
    const size_t row = size_t(sq.q0) + (r.reverse ? sq.nq - 1 - i : i);
    sx[z] = __bfloat162float(r.x.p[row * r.x.row + h * r.x.head + z]);
    sy[z] = __bfloat162float(r.y.p[row * r.y.row + h * r.y.head + z]) * fs_up;
    const float zz = __bfloat162float(r.z.p[row * r.z.row + h * r.z.head + z]);
    __syncthreads();
    float acc = 0.f;
#pragma unroll
    for (int y = 0; y < D; ++y) {
      if (!r.reverse) S[y] = scaled(S[y], l);
      S[y] = fmaf(sy[y], zz, S[y]);
      acc = fmaf(sx[y], S[y], acc);
      if (r.reverse) S[y] = scaled(S[y], l);
    }
    r.out.p[row * r.out.row + h * r.out.head + z] = __float2bfloat16(acc * fs_out);
    __syncthreads();
  }
  if (r.state_out) {
#pragma unroll
    for (int y = 0; y < D; ++y)
      r.state_out[base + (r.state_t ? z * D + y : y * D + z)] = S[y];
  }
}

// One token for each sequence: read the state, decay it, add k v^T, write it
// back and multiply by q.  Bound by the state's bytes.  A thread owns four
// columns of every (threads / (Z / 4))-th row; Z columns of one head's state
// make a CTA.
template <int D, int Z>
__global__ void __launch_bounds__(256) decay_step_kernel(
    RowView q, RowView k, RowView v, const float* __restrict__ log_decay,
    const float* __restrict__ state_in, float* __restrict__ state_out, RowOut o, int H,
    float scale) {
  constexpr int kPerRow = Z / 4, kRows = 256 / kPerRow, kIter = D / kRows;
  __shared__ float4 part[kRows][kPerRow];
  const int i = blockIdx.x / H, h = blockIdx.x % H, t = threadIdx.x;
  const int z = blockIdx.y * Z + (t % kPerRow) * 4, y0 = t / kPerRow;
  const size_t base = (size_t(i) * H + h) * D * D + z;
  float4 s[kIter];
#pragma unroll
  for (int j = 0; j < kIter; ++j)
    s[j] = *reinterpret_cast<const float4*>(state_in + base + size_t(y0 + j * kRows) * D);
  const Factor l = decay_factor(decay_checked(log_decay[h]), 1);
  const uint2 vw = *reinterpret_cast<const uint2*>(v.p + i * v.row + h * v.head + z);
  const float4 vv = make_float4(bf16_lo(vw.x), bf16_hi(vw.x), bf16_lo(vw.y), bf16_hi(vw.y));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int y = y0 + j * kRows;
    const float kk = __bfloat162float(k.p[i * k.row + h * k.head + y]);
    const float qq = __bfloat162float(q.p[i * q.row + h * q.head + y]);
    s[j].x = fmaf(kk, vv.x, scaled(s[j].x, l));
    s[j].y = fmaf(kk, vv.y, scaled(s[j].y, l));
    s[j].z = fmaf(kk, vv.z, scaled(s[j].z, l));
    s[j].w = fmaf(kk, vv.w, scaled(s[j].w, l));
    *reinterpret_cast<float4*>(state_out + base + size_t(y) * D) = s[j];
    acc.x = fmaf(qq, s[j].x, acc.x);
    acc.y = fmaf(qq, s[j].y, acc.y);
    acc.z = fmaf(qq, s[j].z, acc.z);
    acc.w = fmaf(qq, s[j].w, acc.w);
  }
  part[y0][t % kPerRow] = acc;
  __syncthreads();
  if (t < Z) {
    float sum = 0.f;
#pragma unroll 8
    for (int y = 0; y < kRows; ++y) sum += reinterpret_cast<const float*>(&part[y][0])[t];
    o.p[i * o.row + h * o.head + blockIdx.y * Z + t] = __float2bfloat16(sum * scale);
  }
}

}  // namespace

cudaError_t launch_decay_run(const DecayProblem& p, const DecayRun& r, const Seq* seqs,
                             const float* log_decay, int* err, cudaStream_t s) {
  (void)err;
  const dim3 grid(p.n_seq, p.H);
  const float fo = r.reverse ? 1.f : p.scale, fu = r.reverse ? p.scale : 1.f;
  if (p.d == 128)
    decay_run_kernel<128><<<grid, 128, 0, s>>>(r, seqs, log_decay, p.H, fo, fu);
  else
    decay_run_kernel<64><<<grid, 64, 0, s>>>(r, seqs, log_decay, p.H, fo, fu);
  return cudaGetLastError();
}

cudaError_t launch_decay_step(const DecayProblem& p, const void* q, const void* k, const void* v,
                              const float* log_decay, const float* state_in, float* state_out,
                              void* o, cudaStream_t s) {
  using B = __nv_bfloat16;
  const RowView vq{static_cast<const B*>(q), p.q.row, p.q.head},
      vk{static_cast<const B*>(k), p.k.row, p.k.head},
      vv{static_cast<const B*>(v), p.v.row, p.v.head};
  const RowOut vo{static_cast<B*>(o), p.o.row, p.o.head};
  const dim3 grid(p.n_seq * p.H, p.d / 32);
  if (p.d == 128)
    decay_step_kernel<128, 32><<<grid, 256, 0, s>>>(vq, vk, vv, log_decay, state_in, state_out,
                                                    vo, p.H, p.scale);
  else
    decay_step_kernel<64, 32><<<grid, 256, 0, s>>>(vq, vk, vv, log_decay, state_in, state_out, vo,
                                                   p.H, p.scale);
  return cudaGetLastError();
}

}  // namespace sla
