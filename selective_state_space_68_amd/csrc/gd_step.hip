// The gated delta rule, one token: the recurrent form
//     S <- a S;   u = beta (v - S^T k);   S <- S + k u^T;   o = scale S^T q
// for every (sequence, head), with S [K][V] float32 in HBM (a = exp(g)).
//
// The step reads and writes each state once, so it is bound by HBM (a state pool of a few hundred sequences is far
// larger than any cache).  u needs the whole state before any of it changes, so a workgroup holds its state in
// registers between the two (at most 64 floats a thread): S^T k and S^T q are formed together on the way in, and
//     o = scale (a S^T q + (q.k) u)
// needs no second look at the new state.  A lane owns 4 consecutive columns of every `rows`-th row; the rows' parts
// are added up through LDS in one order.  256 sequences of 40 heads, 128 x 128: 259 us, 5.2 TB/s, a copy's rate; one sequence of 24
// heads, 64 x 64: 5.2 us of latency.
#include "device_common.hpp"
#include "lm_kernels.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// CPT: consecutive columns per thread (4: rows of states move as vectors).  N: rows of a thread at most.
template <typename ACT, int CPT, int N>
__global__ __launch_bounds__(kThreads) void gd_step_kernel(GdStepArgs p) {
  __shared__ float sq[kLaMaxDim], sk[kLaMaxDim], su[kLaMaxDim], s_qk;
  __shared__ __attribute__((aligned(16))) float part[2][kThreads * CPT];
  const int tid = threadIdx.x;
  const int K = p.K, V = p.V;
  const uint32_t row_b = blockIdx.x / static_cast<uint32_t>(p.H);   // (32-bit: a 64-bit division is 500 cycles)
  const int64_t bh = blockIdx.x, b = row_b;
  const int h = static_cast<int>(blockIdx.x - row_b * static_cast<uint32_t>(p.H));
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool live = slot >= 0 && slot < p.states;   // (an absent sequence: its output is zero, no state is touched)
  const int64_t o0 = bh * V;
  if (!live) {
    for (int i = tid; i < V; i += kThreads) store_act<ACT>(p.o, o0 + i, 0.0f);
    return;
  }
  const int per_row = V / CPT;                      // threads of a row (CPT is 4 only where it divides V)
  const int rows = kThreads / per_row;              // rows in flight
  const int r0 = tid / per_row, c0 = tid % per_row * CPT;
  const bool mine = r0 < rows;
  const int64_t s0 = ((slot * p.H + h) * K) * V + c0;
  float S[N][CPT];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = r0 + i * rows;
#pragma unroll
    for (int e = 0; e < CPT; ++e) S[i][e] = 0.0f;
    if (mine && r < K) {
      const float* at = p.state_in + s0 + static_cast<int64_t>(r) * V;
      if constexpr (CPT == 4) {
        const float4 x = *reinterpret_cast<const float4*>(at);
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
      } else {
        S[i][0] = *at;
      }
    }
  }
  const int64_t q0 = b * p.qs[0] + (h / p.qdiv) * p.qs[1], k0 = b * p.ks[0] + (h / p.kdiv) * p.ks[1],
                v0 = b * p.vs[0] + (h / p.vdiv) * p.vs[1];
  if (tid < K) sq[tid] = load_act<ACT>(p.q, q0 + tid);
  else if (tid >= 128 && tid - 128 < K) sk[tid - 128] = load_act<ACT>(p.k, k0 + tid - 128);
  const float v = tid < V ? load_act<ACT>(p.v, v0 + tid) : 0.0f;
  const float a = expf(p.g[bh]), beta = p.beta[bh];
  __syncthreads();
  if (tid < 64) {                                   // q.k (a thread that adds it up for itself waits for LDS K times)
    float qk = tid < K ? sq[tid] * sk[tid] : 0.0f;
    if (tid + 64 < K) qk = __builtin_fmaf(sq[tid + 64], sk[tid + 64], qk);
    qk = wave_sum(qk);
    if (tid == 0) s_qk = qk;
  }
  if (mine) {
    float kS[CPT], qS[CPT];
#pragma unroll
    for (int e = 0; e < CPT; ++e) kS[e] = qS[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i * rows;
      if (r >= K) continue;
      const float kv = sk[r], qv = sq[r];
#pragma unroll
      for (int e = 0; e < CPT; ++e) {
        kS[e] = __builtin_fmaf(kv, S[i][e], kS[e]);
        qS[e] = __builtin_fmaf(qv, S[i][e], qS[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < CPT; ++e) {
      part[0][r0 * V + c0 + e] = kS[e];
      part[1][r0 * V + c0 + e] = qS[e];
    }
  }
  __syncthreads();
  if (tid < V) {
    float kS = 0.0f, qS = 0.0f;
    const float qk = s_qk;
    for (int r = 0; r < rows; ++r) {
      kS += part[0][r * V + tid];
      qS += part[1][r * V + tid];
    }
    const float u = beta * __builtin_fmaf(-a, kS, v);
    su[tid] = u;
    store_act<ACT>(p.o, o0 + tid, p.scale * __builtin_fmaf(a, qS, qk * u));
  }
  __syncthreads();
  if (mine) {
    float u[CPT];
#pragma unroll
    for (int e = 0; e < CPT; ++e) u[e] = su[c0 + e];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i * rows;
      if (r >= K) continue;
      const float kv = sk[r];
      float* at = p.state_out + s0 + static_cast<int64_t>(r) * V;
#pragma unroll
      for (int e = 0; e < CPT; ++e) S[i][e] = __builtin_fmaf(a, S[i][e], kv * u[e]);
      if constexpr (CPT == 4) *reinterpret_cast<float4*>(at) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
      else *at = S[i][0];
    }
  }
}

}  // namespace

hipError_t launch_gd_step(const GdStepArgs& a, Dt dt, hipStream_t s) {
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.state_in) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.state_out) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(a.batch * a.H));
  // rows of a thread: 128 / (256 / (V / 4)) = 16 at most by fours, 128 / (256 / V) = 64 by ones
  if (dt == Dt::BF16) {
    if (vec) hipLaunchKernelGGL((gd_step_kernel<ActBF16, 4, 16>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((gd_step_kernel<ActBF16, 1, 64>), grid, dim3(kThreads), 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((gd_step_kernel<ActF32, 4, 16>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((gd_step_kernel<ActF32, 1, 64>), grid, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace ssm
