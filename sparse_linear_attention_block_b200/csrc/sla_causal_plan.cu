// Device-side preparation of the causal operators: the sequences' offsets are
// checked and laid down as one table that the kernels read.
#include "sla_causal.h"
#include "sla_ptx.cuh"

namespace sla {
namespace {

// A sequence whose offsets decrease, leave the tensor or exceed max_q is
// replaced by an empty one and reported.
__global__ void causal_plan_kernel(const int32_t* __restrict__ q_off,
                                   const int32_t* __restrict__ k_off,
                                   const int32_t* __restrict__ k_len, int n_seq, int total_q,
                                   int total_k, int max_q, Seq* __restrict__ seqs, int* err) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n_seq) return;
  const long long q0 = q_off[i], q1 = q_off[i + 1], k0 = k_off[i];
  const long long k1 = k_len ? k0 + k_len[i] : k_off[i + 1];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= total_q && q1 - q0 <= max_q && k0 >= 0 &&
                  k1 >= k0 && k1 <= total_k;
  if (!ok) set_error(err, SLA_ERR_DEVICE);
  seqs[i] = ok ? Seq{int(q0), int(q1 - q0), int(k0), int(k1 - k0)} : Seq{0, 0, 0, 0};
}

__global__ void decay_plan_kernel(const int32_t* __restrict__ off,
                                  const float* __restrict__ log_decay, int n_seq, int total, int H,
                                  Seq* __restrict__ seqs, int* err) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < H && !(log_decay[i] <= 0.f)) set_error(err, SLA_ERR_DEVICE);
  if (i >= n_seq) return;
  const int a = off[i], b = off[i + 1];
  const bool ok = a >= 0 && b >= a && b <= total;
  if (!ok) set_error(err, SLA_ERR_DEVICE);
  // -1 marks a bad sequence: nothing of it is written, not even its state
  seqs[i] = ok ? Seq{a, b - a, 0, 0} : Seq{0, -1, 0, 0};
}

}  // namespace

cudaError_t launch_causal_plan(const CausalProblem& p, const int32_t* q_off, const int32_t* k_off,
                               const int32_t* k_len, Seq* seqs, int* err, cudaStream_t s) {
  causal_plan_kernel<<<(p.n_seq + 255) / 256, 256, 0, s>>>(q_off, k_off, k_len, p.n_seq, p.total_q,
                                                          p.total_k, p.max_q, seqs, err);
  return cudaGetLastError();
}

cudaError_t launch_decay_plan(const DecayProblem& p, const int32_t* off, const float* log_decay,
                              Seq* seqs, int* err, cudaStream_t s) {
  const int n = p.n_seq > p.H ? p.n_seq : p.H;
  decay_plan_kernel<<<(n + 255) / 256, 256, 0, s>>>(off, log_decay, p.n_seq, p.total, p.H, seqs,
                                                    err);
  return cudaGetLastError();
}

}  // namespace sla
