// Linear attention, one token: the recurrent form
//     S <- lam S + k v^T,    o = scale q S
// for every (sequence, head), with S [K][V] float32 in HBM (lam = exp(log_decay)).
//
// The step reads and writes each state once and does 5 flops per entry, so it is bound by
// HBM (a state pool of a few hundred sequences is far larger than any cache).  A workgroup
// owns one state: a lane streams 4 consecutive columns of every `rows`-th row, and the workgroup
// adds up the rows' parts of o through LDS, in one order.
// q and k are read into LDS once as float32.
//
// Measured: 256 sequences of 40 heads, 128 x 128 (1.35 GB read and written): 258 us, 5.2 TB/s, what a copy of
// that size reaches.  One sequence of 24 heads of 64: 4.1 us, the time of a launch and two trips to memory.
#include "device_common.hpp"
#include "lm_kernels.hpp"
#include "scan_common.hpp"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// CPT: consecutive columns per thread (4: rows of states and of v, o move as vectors).
template <typename ACT, int CPT>
__global__ __launch_bounds__(kThreads) void la_step_kernel(LaStepArgs p) {
  __shared__ float sq[kLaMaxDim], sk[kLaMaxDim];
  __shared__ __attribute__((aligned(16))) float so[kThreads * CPT];
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
  const int64_t q0 = b * p.qs[0] + (h / p.qdiv) * p.qs[1], k0 = b * p.ks[0] + (h / p.kdiv) * p.ks[1];
  if (tid < K) sq[tid] = load_act<ACT>(p.q, q0 + tid) * p.scale;
  else if (tid >= 128 && tid - 128 < K) sk[tid - 128] = load_act<ACT>(p.k, k0 + tid - 128);
  const float lam = expf(p.log_decay[h]);
  const int per_row = V / CPT;                      // threads of a row (CPT is 4 only where it divides V)
  const int rows = kThreads / per_row;              // rows in flight
  const int r0 = tid / per_row, c0 = tid % per_row * CPT;
  const int64_t v0 = b * p.vs[0] + (h / p.vdiv) * p.vs[1];
  float vv[CPT], acc[CPT];
#pragma unroll
  for (int e = 0; e < CPT; ++e) {
    vv[e] = load_act<ACT>(p.v, v0 + c0 + e);        // (c0 + e < V always)
    acc[e] = 0.0f;
  }
  __syncthreads();
  const int64_t s0 = ((slot * p.H + h) * K) * V + c0;
  if (r0 < rows) {
#pragma unroll 8
    for (int r = r0; r < K; r += rows) {
      const float qv = sq[r], kv = sk[r];
      const int64_t at = s0 + static_cast<int64_t>(r) * V;
      float s[CPT];
      if constexpr (CPT == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p.state_in + at);
        s[0] = x.x; s[1] = x.y; s[2] = x.z; s[3] = x.w;
      } else {
        s[0] = p.state_in[at];
      }
#pragma unroll
      for (int e = 0; e < CPT; ++e) {
        s[e] = __builtin_fmaf(lam, s[e], kv * vv[e]);
        acc[e] = __builtin_fmaf(qv, s[e], acc[e]);
      }
      if constexpr (CPT == 4) *reinterpret_cast<float4*>(p.state_out + at) = make_float4(s[0], s[1], s[2], s[3]);
      else p.state_out[at] = s[0];
    }
#pragma unroll
    for (int e = 0; e < CPT; ++e) so[(r0 * per_row) * CPT + c0 + e] = acc[e];
  }
  __syncthreads();
  for (int i = tid; i < V; i += kThreads) {
    float s = 0.0f;
    for (int r = 0; r < rows; ++r) s += so[r * per_row * CPT + i];
    store_act<ACT>(p.o, o0 + i, s);
  }
}

}  // namespace

hipError_t launch_la_step(const LaStepArgs& a, Dt dt, hipStream_t s) {
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.state_in) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.state_out) % 16 == 0;
  const dim3 grid(static_cast<unsigned>(a.batch * a.H));
  if (dt == Dt::BF16) {
    if (vec) hipLaunchKernelGGL((la_step_kernel<ActBF16, 4>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((la_step_kernel<ActBF16, 1>), grid, dim3(kThreads), 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((la_step_kernel<ActF32, 4>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((la_step_kernel<ActF32, 1>), grid, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace ssm
