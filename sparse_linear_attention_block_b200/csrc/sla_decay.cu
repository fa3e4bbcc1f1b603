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

// Design of a run (sm_100a).  A CTA (256 threads, two CTAs per SM) walks a piece
// of a sequence in chunks of 64 tokens with the state S^T [z][y] in registers
// (fp32).  Per chunk of r tokens, w_n = l^n, forward (reversed runs mirror the
// exponents):
//   A[s][t]  = y_s . x_t                          MMA, tokens s on the lanes
//   O1[z][t] = sum_y S[z][y] x_t[y]               MMA, S rounded to bf16 in TMEM
//   P[s][t]  = w_{t-s} A[s][t]  (s <= t)          bf16, to shared memory
//   O2[z][t] = sum_s z_s P[s][t]                  MMA
//   U[z][y]  = sum_s z_s w_{r-1-s} y_s            MMA
//   out_t    = w_{t+1} O1[.][t] + O2[.][t],  S = w_r S + U
// The state is held to 32 bits: w y is fed as three bf16 numbers (their sum has
// 24 bits), U starts from 0 in every chunk (the tensor core's sums truncate, a
// running one would drift) and w_r is a two-number factor; only what a query
// reads (S and P as operands) is rounded to bf16, like the output.
// The features lie on the TMEM lanes everywhere (M = 128, for d = 64 with lanes
// that nobody reads), so the state goes into an A operand without leaving its
// lanes.  TMEM: S (bf16), then U at 0, A, then O2 at 128, O1 at 192: 256 columns.
// The bytes of a chunk (x, y, z, out) take longer than its products; what is
// to be hidden is the chain state -> S in bf16 -> products -> state, which two
// CTAs per SM do for one another.  A and O1 run while w y is split, the output
// is written while U runs.
template <int D>
struct DrSmem {
  static constexpr int kT = 64 * D * 2;                      // x, y or z of a chunk
  static constexpr int kX = 0, kY = kT, kZ = 2 * kT, kP = 3 * kT;
  // P, then (when O2 has read it) the chunk's output [t][z] on its way out
  static constexpr int kYs = kP + (8192 > kT ? 8192 : kT);
  static constexpr int kPow = kYs + 3 * kT;   // l^n, n = 0 .. 64 (reversed runs: n = 64 .. 0)
  static constexpr int kMix = kPow + 264;     // 129 factors by t - s + 64: scale l^|t - s| or 0
  static constexpr int kBars = kMix + 520;
  // two CTAs fit on an SM; not more, as each takes half of TMEM
  static constexpr int kTotal = kBars + 96 > 80 * 1024 ? kBars + 96 : 80 * 1024;
  static_assert(kTotal <= (228 * 1024 - 2048) / 2, "two CTAs per SM");
};
struct DrBars {
  Factor carry[2];  // of a whole chunk, of the piece's last one
  uint64_t x_full, y_full, z_full, a_done, o_done, u_done;
  uint32_t tmem_base;
  int abort_flag;
};

struct DrArgs {
  const int* counts;
  const Piece* pieces;
  float* states;
  const float* log_decay;
  DecayRun r;
  int H, most_slots;
  float scale;
  int* err;
};

// The bf16 numbers of the upper halves of two fp32 numbers, and their values.
__device__ __forceinline__ uint32_t upper_halves(float2 x) {
  return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
__device__ __forceinline__ float2 upper_parts(float2 x) {
  return make_float2(bf16_hi(__float_as_uint(x.x)), bf16_hi(__float_as_uint(x.y)));
}

// kStateOnly: the piece's own sum (from a zero state) into its slot, no output.
template <int D, bool kStateOnly>
__global__ void __launch_bounds__(256, 2) decay_run_kernel(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
    const __grid_constant__ CUtensorMap tm_z, const DrArgs g) {
  using L = DrSmem<D>;
  constexpr int kHalf = D / 2;  // state columns of a warpgroup
  extern __shared__ __align__(1024) uint8_t smem[];
  const int idx = blockIdx.x / g.H, h = blockIdx.x % g.H;
  if (kStateOnly ? idx >= g.counts[0]
                 : !(idx < g.counts[0] ||
                     (idx >= g.most_slots && idx - g.most_slots < g.counts[2])))
    return;
  const Piece pc = g.pieces[idx];
  const bool rev = g.r.reverse;
  // the walk over the pieces does not need the last one's sum
  if (kStateOnly && (rev ? pc.first : pc.last)) return;
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) set_error(g.err, SLA_ERR_DEVICE);
    return;
  }
  float* pw = reinterpret_cast<float*>(smem + L::kPow);
  float* mix = reinterpret_cast<float*>(smem + L::kMix);
  DrBars& bb = *reinterpret_cast<DrBars*>(smem + L::kBars);
  int* err = g.err;
  volatile int* abort_flag = &bb.abort_flag;
  const int t = threadIdx.x, warp = t / 32, lane = t % 32;
  const int wg = warp >> 2, z = (warp & 3) * 32 + lane;  // TMEM lane
  const float gl = decay_checked(g.log_decay[h]);

  if (warp == 0) tmem_alloc(&bb.tmem_base, 256);
  if (t == 32) {
    mbar_init(&bb.x_full, 1);
    mbar_init(&bb.y_full, 1);
    mbar_init(&bb.z_full, 1);
    mbar_init(&bb.a_done, 1);
    mbar_init(&bb.o_done, 1);
    mbar_init(&bb.u_done, 1);
    bb.abort_flag = 0;
    fence_barrier_init();
  }
  const int chunks = (pc.rows + 63) / 64, tail = pc.rows - (chunks - 1) * 64;
  // Factors.  Forward: an update has l^{r-1-s}, the state's share of out_t scale l^{t+1}.
  // Reversed: scale l^{s+1}, and l^{r-1-t}.  With l^n in `pw` and scale l^n in `mix` each of
  // them lies in one of the two tables, ascending in t.
  if (t < 129) {
    const int n = rev ? 64 - t : t - 64;  // |t - s| on the visible side
    mix[t] = n >= 0 ? g.scale * decay_factor(gl, n).hi : 0.f;
  } else if (t < 129 + 65) {
    const int n = t - 129;
    pw[rev ? 64 - n : n] = decay_factor(gl, n).hi;
  } else if (t >= 224 && t < 226) {
    bb.carry[t - 224] = decay_factor(gl, t == 224 ? 64 : tail);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem_base;
  const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
  const uint32_t tU = tmem + lane_base + wg * kHalf, tA = tmem + lane_base + 128,
                 tO1 = tmem + lane_base + 192;
  // rows of the c-th chunk in walking order
  auto chunk_row = [&](int c) { return (rev ? chunks - 1 - c : c) * 64; };
  auto load = [&](const CUtensorMap& tm, int at, uint64_t* bar, int c) {  // one thread
    mbar_arrive_expect_tx(bar, L::kT);
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      tma_load_3d(smem + at + k * 8192, bar, &tm, k * 64, pc.row + chunk_row(c), h);
  };
  if (t == 0 && chunks > 0) {
    load(tm_y, L::kY, &bb.y_full, 0);
    if (!kStateOnly) load(tm_x, L::kX, &bb.x_full, 0);
    load(tm_z, L::kZ, &bb.z_full, 0);
  }

  // the state before the piece: a thread keeps kHalf columns of its lane's row
  float2 S[kHalf / 2];
  {
    const size_t dd = size_t(D) * D;
    const float* src = nullptr;
    bool turned = false;
    if (!kStateOnly) {
      if (pc.slot >= 0) {
        src = g.states + (size_t(pc.slot) * g.H + h) * dd;
      } else if (g.r.state_in) {
        src = g.r.state_in + (size_t(pc.seq) * g.H + h) * dd;
        turned = g.r.state_t;
      }
    }
#pragma unroll
    for (int e = 0; e < kHalf; ++e) {
      const int y = wg * kHalf + e;
      const float x = src && z < D ? src[turned ? z * D + y : y * D + z] : 0.f;
      if (e & 1)
        S[e / 2].y = x;
      else
        S[e / 2].x = x;
    }
  }
  // what a query reads: the state rounded to bf16, as an operand over the place of U
  auto put_state = [&]() {
#pragma unroll
    for (int q = 0; q < kHalf / 2; q += 16) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = pack_bf16(S[q + e].x, S[q + e].y);
      tmem_st16(tU + q, w);
    }
    tmem_st_wait();
  };
  // A = Y X^T and O1 = S X^T of chunk c (one thread)
  auto issue_ao = [&](int c) -> bool {
    constexpr uint32_t id_a = idesc_bf16(128, 64, 0, 0);
    if (!mbar_wait(&bb.y_full, c & 1, err, abort_flag) ||
        !mbar_wait(&bb.x_full, c & 1, err, abort_flag))
      return false;
    tc_fence_after();
    const uint64_t yd = desc_kmajor_base(smem_u32(smem + L::kY)),
                   xd = desc_kmajor_base(smem_u32(smem + L::kX));
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      mma_ss(tmem + 128, desc_advance(yd, kmajor_step_bytes(64, ks)),
             desc_advance(xd, kmajor_step_bytes(64, ks)), id_a, ks > 0);
    constexpr int kPer = D / 32;  // k-steps of a warpgroup's half of the state
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      mma_ts(tmem + 192, tmem + (ks / kPer) * kHalf + (ks % kPer) * 8,
             desc_advance(xd, kmajor_step_bytes(64, ks)), id_a, ks > 0);
    mma_commit(&bb.a_done);
    return true;
  };
  bool ok = true;
  if (!kStateOnly && chunks > 0) {
    put_state();
    tc_fence_before();
    __syncthreads();
    if (t == 0) ok = issue_ao(0);
    __syncwarp();
  }

  for (int c = 0; c < chunks; ++c) {
    const int row0 = chunk_row(c), r = min(64, pc.rows - row0);
    const uint32_t ph = c & 1;
    const bool more = c + 1 < chunks;
    ok = mbar_wait(&bb.y_full, ph, err, abort_flag) && ok;
    if (ok) {
      // w y in three bf16 parts; rows behind the piece are 0
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int e = t + i * 256, s = e / (D / 8), col = (e % (D / 8)) * 8;
        const uint32_t at = (col >> 6) * 8192 + sw128_offset(s, col & 63);
        const uint4 u = *reinterpret_cast<const uint4*>(smem + L::kY + at);
        // 24 bits of the product in three parts: the upper halves of the number, of what is
        // left, and the rest rounded
        const float f = rev ? mix[63 - s] : pw[s < r ? r - 1 - s : 0];
        const bool in = s < r;
        const uint32_t w[4] = {in ? u.x : 0u, in ? u.y : 0u, in ? u.z : 0u, in ? u.w : 0u};
        uint32_t p0[4], p1[4], p2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float2 x = __fmul2_rn(make_float2(bf16_lo(w[k]), bf16_hi(w[k])), make_float2(f, f));
          p0[k] = upper_halves(x);
          x = __ffma2_rn(upper_parts(x), make_float2(-1.f, -1.f), x);
          p1[k] = upper_halves(x);
          x = __ffma2_rn(upper_parts(x), make_float2(-1.f, -1.f), x);
          p2[k] = pack_bf16(x.x, x.y);
        }
        uint8_t* dst = smem + L::kYs + at;
        *reinterpret_cast<uint4*>(dst) = make_uint4(p0[0], p0[1], p0[2], p0[3]);
        *reinterpret_cast<uint4*>(dst + L::kT) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
        *reinterpret_cast<uint4*>(dst + 2 * L::kT) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
      }
    }
    if (!kStateOnly) {
      ok = ok && mbar_wait(&bb.a_done, ph, err, abort_flag);
      tc_fence_after();
      if (ok && (warp & 3) < 2) {
        const int s = z;
        float v[32];
        tmem_ld32(tA + wg * 32, v);
        tmem_ld_wait();
        const float* f = mix + 64 + wg * 32 - s;
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= f[e];
        if (s >= r) {  // a row of y behind the piece
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st_sw128_unit(smem + L::kP, 64, s, wg * 32 + u * 8,
                        make_uint4(pack_bf16(v[u * 8], v[u * 8 + 1]),
                                   pack_bf16(v[u * 8 + 2], v[u * 8 + 3]),
                                   pack_bf16(v[u * 8 + 4], v[u * 8 + 5]),
                                   pack_bf16(v[u * 8 + 6], v[u * 8 + 7])));
      }
    }
    if (r < 64 && ok && (ok = mbar_wait(&bb.z_full, ph, err, abort_flag))) {
      // the rows of z behind the piece belong to others: 0 times NaN would be NaN
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        for (int b = r * 128 + t * 16; b < 8192; b += 4096)
          *reinterpret_cast<uint4*>(smem + L::kZ + k * 8192 + b) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    ok = __syncthreads_and(ok);
    tc_fence_after();
    if (!ok) break;
    if (t == 32 && more) {  // A, O1 and the split have read y and x
      load(tm_y, L::kY, &bb.y_full, c + 1);
      if (!kStateOnly) load(tm_x, L::kX, &bb.x_full, c + 1);
    }
    if (t == 0) {
      constexpr uint32_t id_o2 = idesc_bf16(128, 64, 1, 1), id_u = idesc_bf16(128, D, 1, 1);
      const uint64_t zd = desc_mnmajor_base(smem_u32(smem + L::kZ), 64);
      ok = mbar_wait(&bb.z_full, ph, err, abort_flag);
      tc_fence_after();
      if (!kStateOnly) {
        const uint64_t pd = desc_mnmajor_base(smem_u32(smem + L::kP), 64);
        if (ok) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss(tmem + 128, desc_advance(zd, mnmajor_step_bytes(ks)),
                   desc_advance(pd, mnmajor_step_bytes(ks)), id_o2, ks > 0);
        }
        mma_commit(&bb.o_done);
      }
      if (ok) {
#pragma unroll
        for (int q = 2; q >= 0; --q) {  // the small parts first
          const uint64_t yd = desc_mnmajor_base(smem_u32(smem + L::kYs + q * L::kT), 64);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss(tmem, desc_advance(zd, mnmajor_step_bytes(ks)),
                   desc_advance(yd, mnmajor_step_bytes(ks)), id_u, q < 2 || ks > 0);
        }
      }
      mma_commit(&bb.u_done);
    }
    __syncwarp();
    if (!kStateOnly) {
      ok = mbar_wait(&bb.o_done, ph, err, abort_flag) && ok;
      tc_fence_after();
      // a warpgroup's 32 tokens: turned in shared memory, out as 16 bytes per thread
      __nv_bfloat16* turn = reinterpret_cast<__nv_bfloat16*>(smem + L::kP) + wg * 32 * D;
      if (ok && (warp & 3) * 32 < D) {
#pragma unroll
        for (int c0 = 0; c0 < 32; c0 += 16) {
          float o1[16], o2[16];
          tmem_ld16(tO1 + wg * 32 + c0, o1);
          tmem_ld16(tA + wg * 32 + c0, o2);
          tmem_ld_wait();
          // (tokens behind the piece get any factor: they are not stored)
          const float* f = (rev ? pw + 65 - r : mix + 65) + wg * 32 + c0;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 x = __ffma2_rn(make_float2(o1[e], o1[e + 1]), make_float2(f[e], f[e + 1]),
                                        make_float2(o2[e], o2[e + 1]));
            const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
            turn[(c0 + e) * D + z] = b.x;
            turn[(c0 + e + 1) * D + z] = b.y;
          }
        }
      }
      named_bar_sync(1 + wg, 128);
      if (ok) {
        __nv_bfloat16* dst =
            g.r.out.p + (size_t(pc.row) + row0 + wg * 32) * g.r.out.row + h * g.r.out.head;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int e = (t & 127) + i * 128, k = e / (D / 8), col = (e % (D / 8)) * 8;
          if (wg * 32 + k < r)
            *reinterpret_cast<uint4*>(dst + k * g.r.out.row + col) =
                *reinterpret_cast<const uint4*>(turn + k * D + col);
        }
      }
    }
    ok = mbar_wait(&bb.u_done, ph, err, abort_flag) && ok;
    tc_fence_after();
    if (t == 32 && ok && more) load(tm_z, L::kZ, &bb.z_full, c + 1);
    __syncwarp();
    // S = w_r S + U
    const Factor carry = bb.carry[r < 64];
    const float2 hi = make_float2(carry.hi, carry.hi), lo = make_float2(carry.lo, carry.lo);
#pragma unroll
    for (int c0 = 0; c0 < kHalf; c0 += 16) {
      float v[16];
      tmem_ld16(tU + c0, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2& x = S[c0 / 2 + e];
        x = __ffma2_rn(x, hi, __ffma2_rn(x, lo, make_float2(v[2 * e], v[2 * e + 1])));
      }
    }
    if (!kStateOnly && more) put_state();
    tc_fence_before();
    ok = __syncthreads_and(ok);
    tc_fence_after();
    if (!ok) break;
    if (!kStateOnly && more && t == 0) ok = issue_ao(c + 1);
    __syncwarp();
  }

  if (!ok) {
    // let copies and products already in flight end before the CTA exits (a barrier
    // without one runs into its time limit)
    if (t == 0) {
      for (uint32_t q = 0; q < 2; ++q) {
        mbar_wait(&bb.x_full, q, nullptr, nullptr);
        mbar_wait(&bb.y_full, q, nullptr, nullptr);
        mbar_wait(&bb.z_full, q, nullptr, nullptr);
        mbar_wait(&bb.u_done, q, nullptr, nullptr);
      }
    }
  } else if (kStateOnly || (g.r.state_out && (rev ? pc.first : pc.last))) {
    float* dst = kStateOnly ? g.states + (size_t(pc.slot) * g.H + h) * D * D
                            : g.r.state_out + (size_t(pc.seq) * g.H + h) * D * D;
if (z < D) {
#pragma unroll
      for (int e = 0; e < kHalf; ++e)
        dst[size_t(wg * kHalf + e) * D + z] = e & 1 ? S[e / 2].y : S[e / 2].x;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_free(tmem, 256);
}

// The states before the pieces of the cut sequences, over their sums: with U_j
// the j-th piece's sum and n_j its rows,  S_0 = state_in,  S_{j+1} = l^{n_j} S_j + U_j.
// Four elements per thread.
template <int D>
__global__ void __launch_bounds__(256) decay_scan_kernel(const int* __restrict__ counts,
                                                         const Split* __restrict__ splits,
                                                         float* __restrict__ states,
                                                         const float* __restrict__ log_decay,
                                                         DecayRun r, int H, int rows) {
  if (int(blockIdx.x) >= counts[1]) return;
  const Split sp = splits[blockIdx.x];
  const int h = blockIdx.y, e = (blockIdx.z * 256 + threadIdx.x) * 4;
  const float gl = decay_checked(log_decay[h]);
  const Factor full = decay_factor(gl, rows), part = decay_factor(gl, sp.last_rows);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r.state_in) {
    const float* p = r.state_in + (size_t(sp.seq) * H + h) * D * D;
    const int y = e / D, z = e % D;
    s = r.state_t ? make_float4(p[z * D + y], p[(z + 1) * D + y], p[(z + 2) * D + y],
                                p[(z + 3) * D + y])
                  : *reinterpret_cast<const float4*>(p + e);
  }
  const auto at = [&](int j) {
    const int k = r.reverse ? sp.pieces - 1 - j : j;
    return reinterpret_cast<float4*>(states + (size_t(sp.slot + k) * H + h) * D * D + e);
  };
  constexpr int kBatch = 8;  // sums in flight (38 us with one, see the run's figures)
  for (int j0 = 0; j0 < sp.pieces; j0 += kBatch) {
    float4 u[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (j0 + b < sp.pieces - 1) u[b] = *at(j0 + b);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int j = j0 + b;
      if (j >= sp.pieces) break;
      *at(j) = s;
      if (j == sp.pieces - 1) break;  // nobody asks for the state behind the last piece
      const Factor f = r.reverse && j == 0 ? part : full;
      s = make_float4(scaled(s.x, f) + u[b].x, scaled(s.y, f) + u[b].y, scaled(s.z, f) + u[b].z,
                      scaled(s.w, f) + u[b].w);
    }
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

namespace {

template <int D, bool kStateOnly>
cudaError_t run(const DecayProblem& p, const DecayCut& cut, const DecayRun& r, const DecayLists& l,
                const float* log_decay, int* err, cudaStream_t s) {
  const auto map = [&](CUtensorMap* m, const RowView& v) {
    return make_tmap_rows(m, v.p, p.total, p.H, D, sla_strides{v.row, v.head}, 64);
  };
  CUtensorMap tx, ty, tz;
  if (!map(&tx, r.x) || !map(&ty, r.y) || !map(&tz, r.z)) return cudaErrorInvalidValue;
  const DrArgs a{l.counts,       l.pieces, l.states,
                 log_decay,      r,        p.H,
                 cut.most_slots, p.scale, err};
  auto* kernel = decay_run_kernel<D, kStateOnly>;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DrSmem<D>::kTotal);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(cut.most_slots + (kStateOnly ? 0 : p.n_seq)) * p.H;
  kernel<<<grid, 256, DrSmem<D>::kTotal, s>>>(tx, ty, tz, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_run(const DecayProblem& p, const DecayCut& cut, const DecayRun& r,
                             const DecayLists& l, const float* log_decay, int* err,
                             cudaStream_t s) {
  return p.d == 128 ? run<128, false>(p, cut, r, l, log_decay, err, s)
                    : run<64, false>(p, cut, r, l, log_decay, err, s);
}

cudaError_t launch_decay_pieces(const DecayProblem& p, const DecayCut& cut, const DecayRun& r,
                                const DecayLists& l, const float* log_decay, int* err,
                                cudaStream_t s) {
  return p.d == 128 ? run<128, true>(p, cut, r, l, log_decay, err, s)
                    : run<64, true>(p, cut, r, l, log_decay, err, s);
}

cudaError_t launch_decay_scan(const DecayProblem& p, const DecayCut& cut, const DecayRun& r,
                              const DecayLists& l, const float* log_decay, cudaStream_t s) {
  const dim3 grid(cut.most_splits, p.H, p.d * p.d / 1024);
  if (p.d == 128)
    decay_scan_kernel<128><<<grid, 256, 0, s>>>(l.counts, l.splits, l.states, log_decay, r, p.H,
                                                cut.rows);
  else
    decay_scan_kernel<64><<<grid, 256, 0, s>>>(l.counts, l.splits, l.states, log_decay, r, p.H,
                                               cut.rows);
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
